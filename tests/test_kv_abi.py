"""The quantized K/V cache calls without a GPU: sizes, structures and
refusals.  Every refused call returns before any HIP call; the device
addresses are fake and never touched."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from error_compensated_bit_amd import binding as B
from error_compensated_bit_amd import sim

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000
GOOD_CACHE = dict(bits=4, group=128, head_dim=128, kv_heads=2, page_size=16, reserved=0, num_pages=4,
                  k_codes=A, v_codes=A, k_params=A, v_params=A)
GOOD_BATCH = dict(seqs=2, rows=6, max_new=4, max_len=64, table_stride=4, row_start=A, kv_len=A, page_table=A)
GOOD_ROWS = dict(data=A, row_stride=256, head_stride=128, dtype=B.ECHO_KV_BF16, reserved=0)
Q_ROWS = dict(GOOD_ROWS, row_stride=512)


def ref(cls, good, **kw):
    return ctypes.byref(cls(**{**good, **kw}))


def cache(**kw):
    return ref(B.echo_kv_cache, GOOD_CACHE, **kw)


def batch(**kw):
    return ref(B.echo_kv_batch, GOOD_BATCH, **kw)


def rows(**kw):
    return ref(B.echo_kv_rows, GOOD_ROWS, **kw)


def qrows(**kw):
    return ref(B.echo_kv_rows, Q_ROWS, **kw)


def attention(L, c=None, b=None, heads=4, q=None, out=None, scale=0.1, causal=1, window=0, sinks=0, ws=None, n=0):
    return L.echo_kv_attention(c or cache(), b or batch(), heads, q or qrows(), out or qrows(), scale, causal, window,
                               sinks, ws, n, None)


CACHE_FAULTS = [
    (dict(bits=5), B.ECHO_ERR_ARG), (dict(bits=0), B.ECHO_ERR_ARG), (dict(group=16), B.ECHO_ERR_ARG),
    (dict(group=48), B.ECHO_ERR_ARG), (dict(head_dim=96), B.ECHO_ERR_ARG), (dict(head_dim=64), B.ECHO_ERR_ARG),
    (dict(head_dim=512), B.ECHO_ERR_ARG), (dict(kv_heads=0), B.ECHO_ERR_ARG), (dict(kv_heads=4097), B.ECHO_ERR_ARG),
    (dict(page_size=8), B.ECHO_ERR_ARG), (dict(page_size=48), B.ECHO_ERR_ARG), (dict(page_size=512), B.ECHO_ERR_ARG),
    (dict(num_pages=0), B.ECHO_ERR_SHAPE), (dict(num_pages=1 << 31), B.ECHO_ERR_SHAPE),
    (dict(k_codes=None), B.ECHO_ERR_ARG), (dict(v_params=None), B.ECHO_ERR_ARG),
    (dict(v_codes=A + 8), B.ECHO_ERR_ALIGN), (dict(k_params=A + 4), B.ECHO_ERR_ALIGN),
]
BATCH_FAULTS = [
    (dict(seqs=-1), B.ECHO_ERR_SHAPE), (dict(seqs=65536), B.ECHO_ERR_SHAPE), (dict(rows=-1), B.ECHO_ERR_SHAPE),
    (dict(rows=(1 << 30) + 1), B.ECHO_ERR_SHAPE), (dict(max_new=-1), B.ECHO_ERR_SHAPE),
    (dict(max_len=-1), B.ECHO_ERR_SHAPE), (dict(max_len=(1 << 30) + 1), B.ECHO_ERR_SHAPE),
    (dict(table_stride=-1), B.ECHO_ERR_SHAPE), (dict(row_start=None), B.ECHO_ERR_ARG),
    (dict(kv_len=None), B.ECHO_ERR_ARG), (dict(page_table=None), B.ECHO_ERR_ARG),
    (dict(kv_len=A + 2), B.ECHO_ERR_ALIGN),
]
ROWS_FAULTS = [
    (dict(data=None), B.ECHO_ERR_ARG), (dict(data=A + 8), B.ECHO_ERR_ALIGN), (dict(row_stride=257), B.ECHO_ERR_ALIGN),
    (dict(head_stride=132), B.ECHO_ERR_ALIGN), (dict(row_stride=-256), B.ECHO_ERR_ARG),
    (dict(row_stride=1 << 41), B.ECHO_ERR_ARG), (dict(dtype=3), B.ECHO_ERR_ARG), (dict(dtype=-1), B.ECHO_ERR_ARG),
]


@pytest.mark.parametrize("fault,code", CACHE_FAULTS)
def test_cache_faults(fault, code):
    L = B.load_library()
    assert L.echo_kv_write(cache(**fault), batch(), rows(), rows(), None) == code
    assert L.echo_kv_read(cache(**fault), batch(), rows(), rows(), None) == code
    assert attention(L, c=cache(**fault)) == code


@pytest.mark.parametrize("fault,code", BATCH_FAULTS)
def test_batch_faults(fault, code):
    L = B.load_library()
    assert L.echo_kv_write(cache(), batch(**fault), rows(), rows(), None) == code
    assert L.echo_kv_read(cache(), batch(**fault), rows(), rows(), None) == code
    assert attention(L, b=batch(**fault)) == code


@pytest.mark.parametrize("fault,code", ROWS_FAULTS)
def test_rows_faults(fault, code):
    L = B.load_library()
    if "dtype" not in fault:
        assert L.echo_kv_write(cache(), batch(), rows(**fault), rows(), None) == code
        assert L.echo_kv_read(cache(), batch(), rows(), rows(**fault), None) == code
    assert L.echo_kv_write(cache(), batch(), rows(**fault), rows(**fault), None) == code
    assert attention(L, q=qrows(**fault), out=qrows(**fault)) == code


@pytest.mark.parametrize("call,code", [
    (lambda L: L.echo_kv_write(None, batch(), rows(), rows(), None), B.ECHO_ERR_ARG),
    (lambda L: L.echo_kv_write(cache(), None, rows(), rows(), None), B.ECHO_ERR_ARG),
    (lambda L: L.echo_kv_write(cache(), batch(), None, rows(), None), B.ECHO_ERR_ARG),
    (lambda L: L.echo_kv_read(cache(), batch(), rows(), None, None), B.ECHO_ERR_ARG),
    # keys and values of two types
    (lambda L: L.echo_kv_write(cache(), batch(), rows(dtype=B.ECHO_KV_F16), rows(), None), B.ECHO_ERR_ARG),
    # rows that are written may not overlap; rows that are read may
    (lambda L: L.echo_kv_read(cache(), batch(), rows(row_stride=128), rows(), None), B.ECHO_ERR_ARG),
    (lambda L: L.echo_kv_read(cache(), batch(), rows(head_stride=64), rows(), None), B.ECHO_ERR_ARG),
    (lambda L: L.echo_kv_read(cache(), batch(), rows(row_stride=0), rows(), None), B.ECHO_ERR_ARG),
    # more rows than one dispatch covers
    (lambda L: L.echo_kv_write(cache(kv_heads=4096), batch(rows=1 << 30), rows(), rows(), None), B.ECHO_ERR_SHAPE),
    (lambda L: attention(L, heads=3), B.ECHO_ERR_ARG),
    (lambda L: attention(L, heads=0), B.ECHO_ERR_ARG),
    (lambda L: attention(L, heads=1), B.ECHO_ERR_ARG),
    (lambda L: attention(L, scale=float("nan")), B.ECHO_ERR_ARG),
    (lambda L: attention(L, scale=float("inf")), B.ECHO_ERR_ARG),
    (lambda L: attention(L, causal=2), B.ECHO_ERR_ARG),
    (lambda L: attention(L, window=-1), B.ECHO_ERR_ARG),
    (lambda L: attention(L, window=8, sinks=-1), B.ECHO_ERR_ARG),
    (lambda L: attention(L, sinks=4), B.ECHO_ERR_ARG),                       # first keys without a window
    (lambda L: attention(L, causal=0, window=8), B.ECHO_ERR_ARG),
    (lambda L: attention(L, q=qrows(dtype=B.ECHO_KV_F32), out=qrows(dtype=B.ECHO_KV_F32)), B.ECHO_ERR_ARG),
    (lambda L: attention(L, q=qrows(dtype=B.ECHO_KV_F16)), B.ECHO_ERR_ARG),  # q and out of two types
    (lambda L: attention(L, out=qrows(row_stride=256)), B.ECHO_ERR_ARG),
    # the split results need a workspace
    (lambda L: attention(L, b=batch(max_len=65536)), B.ECHO_ERR_ARG),
    (lambda L: attention(L, b=batch(max_len=65536), ws=A + 4, n=1 << 30), B.ECHO_ERR_ALIGN),
    (lambda L: attention(L, b=batch(max_len=65536), ws=A, n=64), B.ECHO_ERR_ARG),
])
def test_refusals(call, code):
    assert call(B.load_library()) == code


def test_calls_without_rows_do_nothing():
    """No rows or no sequences: accepted, and no buffer is looked at."""
    L = B.load_library()
    none = ref(B.echo_kv_rows, dict(data=None, row_stride=0, head_stride=0, dtype=0, reserved=0))
    for b in (batch(rows=0, row_start=None, kv_len=None, page_table=None), batch(seqs=0, row_start=None)):
        assert L.echo_kv_write(cache(k_codes=None), b, none, none, None) == B.ECHO_OK
        assert L.echo_kv_read(cache(), b, none, none, None) == B.ECHO_OK
        assert attention(L, b=b, q=none, out=none) == B.ECHO_OK
    assert attention(L, b=batch(max_new=0), q=none, out=none) == B.ECHO_OK


def test_sizes():
    assert B.echo_kv_codes_bytes(10, 64, 8, 128) == 10 * 64 * 8 * 64
    assert B.echo_kv_codes_bytes(10, 64, 8, 128, bits=8) == 10 * 64 * 8 * 128
    assert B.echo_kv_params_bytes(10, 64, 8, 128) == 10 * 64 * 8 * 4
    assert B.echo_kv_params_bytes(10, 64, 8, 256, group=32) == 10 * 64 * 8 * 32
    assert B.echo_kv_codes_bytes(1 << 30, 256, 4096, 256, bits=8) == 1 << 58   # no 32-bit product
    for bad in (dict(page_size=24), dict(head_dim=80), dict(group=256), dict(bits=2), dict(num_pages=0)):
        kw = dict(num_pages=10, page_size=64, kv_heads=8, head_dim=128, **{})
        kw.update(bad)
        assert B.echo_kv_codes_bytes(**kw) == 0 and B.echo_kv_params_bytes(**kw) == 0
        with pytest.raises(ValueError):
            B.alloc_kv_cache(**kw, device="cpu")


def test_workspace_depends_on_the_sizes_only():
    """Short calls need none; a long one holds 256 counters and D + 2 floats for every row and split."""
    L = B.load_library()

    def size(b, heads=4, causal=1, window=0, sinks=0, c=None):
        return L.echo_kv_workspace_bytes(c or cache(), b, heads, causal, window, sinks)

    assert size(batch()) == 0
    big = size(batch(max_len=65536))
    assert big > 1024 and (big - 1024) % (130 * 4) == 0
    assert big == size(batch(max_len=65536, row_start=None, kv_len=None, page_table=None))
    assert size(batch(max_len=65536, rows=0)) == 0
    assert size(batch(max_len=65536), heads=3) == 0
    assert size(batch(max_len=65536), window=64, sinks=4) < big     # a window leaves little to split
    # enough rows fill the machine without splitting
    assert size(batch(seqs=4096, rows=4096, max_new=1, max_len=2048)) == 0


def test_structures_match_the_header(tmp_path):
    """Sizes and offsets as a C compiler sees them."""
    names = {"echo_kv_cache": B.echo_kv_cache, "echo_kv_batch": B.echo_kv_batch, "echo_kv_rows": B.echo_kv_rows}
    lines = [f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));' for s, c in names.items() for f, _ in c._fields_]
    lines += [f'printf("{s} %zu\\n", sizeof({s}));' for s in names]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "echo.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    for s, c in names.items():
        assert int(got[s]) == ctypes.sizeof(c)
        for f, _ in c._fields_:
            assert int(got[f"{s}.{f}"]) == getattr(c, f).offset


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "echo.h")).read()
    for name in ("ECHO_KV_BF16", "ECHO_KV_F16", "ECHO_KV_F32"):
        m = re.search(rf"#define\s+{name}\s+(-?\d+)", text)
        assert m and int(m.group(1)) == getattr(B, name)


def test_binding_refuses_what_the_library_cannot_see():
    """Types, shapes and devices of tensors; nothing reaches the library."""
    c = B.alloc_kv_cache(4, 16, 2, 128, device="cpu")
    b = B.KVBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                  torch.zeros(2, 4, dtype=torch.int32), rows=6, max_new=4, max_len=64)
    k = torch.zeros(6, 2, 128, dtype=torch.bfloat16)
    q = torch.zeros(6, 4, 128, dtype=torch.bfloat16)
    for call in (lambda: B.echo_kv_write(c, b, k, k, stream=0), lambda: B.echo_kv_read(c, b, k, k, stream=0),
                 lambda: B.prepare_kv_attention(c, b, q, q, 0.1, stream=0)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for t in (k.int(), k[:5], k[:, :1], torch.zeros(6, 2, 64, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="expected"):
            B._kv_rows(t, "k", 6, 2, 128, torch.device("cpu"))
    with pytest.raises(ValueError, match="contiguous"):
        B._kv_rows(torch.zeros(6, 2, 256, dtype=torch.bfloat16)[..., ::2], "k", 6, 2, 128, torch.device("cpu"))
    good = b.desc(torch.device("cpu"))
    assert (good.seqs, good.rows, good.table_stride) == (2, 6, 4)
    for bad in (B.KVBatch(b.row_start.long(), b.kv_len, b.page_table, 6, 4, 64),
                B.KVBatch(b.row_start[:2], b.kv_len, b.page_table, 6, 4, 64),
                B.KVBatch(b.row_start, b.kv_len, b.page_table[:1], 6, 4, 64),
                B.KVBatch(b.row_start, b.kv_len, b.page_table.reshape(-1), 6, 4, 64)):
        with pytest.raises(ValueError):
            bad.desc(torch.device("cpu"))
    with pytest.raises(ValueError, match="k_params"):
        B.KVCache(4, 64, 128, c.k_codes, c.v_codes, c.k_params, c.v_params).desc()


def test_binding_refuses_views_whose_strides_it_cannot_pass_on():
    c = B.alloc_kv_cache(4, 16, 2, 128, device="cpu")
    wide = B.alloc_kv_cache(4, 32, 2, 128, device="cpu")
    b = B.KVBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                  torch.zeros(2, 4, dtype=torch.int32), rows=6, max_new=4, max_len=64)
    for bad in (B.KVBatch(b.row_start, b.kv_len, torch.zeros(2, 8, dtype=torch.int32)[:, :4], 6, 4, 64),
                B.KVBatch(b.row_start, torch.zeros(4, dtype=torch.int32)[::2], b.page_table, 6, 4, 64),
                B.KVBatch(torch.zeros(6, dtype=torch.int32)[::2], b.kv_len, b.page_table, 6, 4, 64)):
        with pytest.raises(ValueError, match="contiguous"):
            bad.desc(torch.device("cpu"))
    with pytest.raises(ValueError, match="v_codes must be contiguous"):
        B.KVCache(4, 128, 128, c.k_codes, wide.v_codes[:, :, :16], c.k_params, c.v_params).desc()


def test_attention_site_refuses_a_batch_that_is_not_the_messages():
    rows, hidden = 6, 32
    a = sim.AttentionRanks([None, None], [torch.zeros(128, hidden)] * 2, None, [torch.zeros(rows, 1, 128)] * 2,
                           [torch.zeros(rows, hidden)] * 2)
    batch = B.KVBatch(None, None, None, rows, rows, rows)
    x = [torch.zeros(rows, 1, 128)] * 2
    for r, b, q in ((sim.Ranks(2, rows * hidden + 1, [], [], [], None), batch, x),
                    (sim.Ranks(2, rows * hidden, [], [], [], None), batch, x[:1]),
                    (sim.Ranks(3, rows * hidden, [], [], [], None), batch, x),
                    (sim.Ranks(2, 7 * hidden, [], [], [], None), B.KVBatch(None, None, None, 7, 7, 7), x)):
        with pytest.raises(ValueError):
            sim.attention_site(None, r, a, b, q, x, x, 0.1)
