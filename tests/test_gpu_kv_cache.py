"""Writing rows into the quantized K/V cache and reading them back, against the
quantizer's definition in 64 bits (codes, steps and zeros bit for bit)."""
import numpy as np
import pytest
import torch

import kv_testutil as U
import oracle as O
from error_compensated_bit_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMS = [(bits, D, G) for bits in (4, 8) for D in (64, 128, 256) for G in (32, 64, 128) if G <= D]


def make_cache(lay, heads, D, bits, group, fill=None):
    c = B.alloc_kv_cache(lay.pages, lay.page, heads, D, bits, group, DEV)
    if fill is not None:
        for t in (c.k_codes, c.v_codes, c.k_params, c.v_params):
            t.view(torch.uint8).fill_(fill)
    return c


def check_written(cache, lay, new, k, v, fill):
    """Every written slot holds the definition's codes and parameters, every
    other byte still the sentinel."""
    rows = U.cache_rows(cache)
    touched = np.zeros((lay.pages, lay.page), bool)
    at = 0
    for b, n in enumerate(new):
        pos = np.arange(lay.lens[b] - n, lay.lens[b])
        page, slot = lay.slots(b, pos)
        touched[page, slot] = True
        for x, (codes, step, zero) in ((k, rows[0]), (v, rows[1])):
            want = U.quantize(U.host64(x[at:at + n]), cache.bits, cache.group)
            assert np.array_equal(codes[page, :, slot], want[0])
            assert np.array_equal(step[page, :, slot], want[1])
            assert np.array_equal(zero[page, :, slot], want[2])
        at += n
    for t in (cache.k_codes, cache.v_codes, cache.k_params, cache.v_params):
        raw = t.contiguous().view(torch.uint8).cpu().numpy().reshape(lay.pages, cache.kv_heads, lay.page, -1)
        assert (raw.transpose(0, 2, 1, 3)[~touched] == fill).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bits,D,G", FORMS)
def test_write_and_read_every_form(bits, D, G, dtype):
    """Ragged sequences (one with no new row, one of a single row), odd head
    count, pages that end inside a run of rows; then rows of a middle part."""
    lay = U.Layout(lens=[37, 5, 1, 64], new=[21, 0, 1, 64], page=16, seed=D + G)
    heads = 3
    cache = make_cache(lay, heads, D, bits, G, fill=0xA5)
    k = U.draw((lay.rows, heads, D), 1, dtype, 3.0, 0.5).to(DEV)
    v = U.draw((lay.rows, heads, D), 2, dtype, 0.01).to(DEV)
    B.echo_kv_write(cache, lay.batch(), k, v)
    torch.cuda.synchronize()
    check_written(cache, lay, lay.new, k, v, 0xA5)
    for out_type in ("bf16", "f16", "f32"):
        back = [torch.full((lay.rows, heads, D), 7.0, dtype=U.DTYPES[out_type], device=DEV) for _ in "kv"]
        B.echo_kv_read(cache, lay.batch(), *back)
        for x, got in ((k, back[0]), (v, back[1])):
            want = U.values(*U.quantize(U.host64(x), bits, G), G)
            want = torch.from_numpy(want.astype(np.float32)).to(U.DTYPES[out_type])
            assert torch.equal(got.cpu(), want)


def test_codes_are_the_all_reduce_quantizers():
    """The same codes, steps and zeros as the all-reduce's quantizer (its C
    oracle) for rows with ties, constants, huge, subnormal and negative zeros."""
    D, G, bits = 128, 128, 4
    x = U.draw((24, 1, D), 5, "f32", 2.0)
    x[1] = 3.25
    x[2] = 0.0
    x[3] = -0.0
    x[4] *= 1e30
    x[5] *= 1e-7
    x[6] = torch.arange(D).remainder(16).float()
    x[7] = (torch.arange(D).remainder(31).float() + 0.5) / 2
    lay = U.Layout([24], [24], 32)
    cache = make_cache(lay, 1, D, bits, G)
    B.echo_kv_write(cache, lay.batch(), x.to(DEV), x.to(DEV))
    (codes, step, zero), _ = U.cache_rows(cache)
    page, slot = lay.slots(0, np.arange(24))
    for i in range(24):
        c, s, z, _ = O.quantize_group(x[i, 0].numpy(), bits)
        assert np.array_equal(codes[page[i], 0, slot[i]], np.asarray(c))
        s, z = np.array([s, z], np.uint16).view(np.float16).astype(np.float64)
        assert step[page[i], 0, slot[i], 0] == s and zero[page[i], 0, slot[i], 0] == z


def test_special_values_leave_finite_parameters():
    """NaN is code 0, infinities the ends of the range, and no parameter in the
    cache is ever NaN or infinite."""
    D = 64
    x = U.draw((6, 2, D), 9, "f32")
    x[0, 0, 3] = float("nan")
    x[1, 0, :] = float("nan")
    x[2, 1, 5] = float("inf")
    x[3, 1, 9] = -float("inf")
    x[4, 0, 0], x[4, 0, 1] = float("inf"), -float("inf")
    x[5, 1] = 3.0e38
    for bits in (4, 8):
        lay = U.Layout([6], [6], 16)
        cache = make_cache(lay, 2, D, bits, 32, fill=0)
        B.echo_kv_write(cache, lay.batch(), x.to(DEV), x.to(DEV))
        check_written(cache, lay, lay.new, x, x, 0)
        for _, step, zero in U.cache_rows(cache):
            assert np.isfinite(step).all() and np.isfinite(zero).all()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_appending_token_by_token_equals_writing_at_once(page):
    """A prompt, then one token per sequence and call: the same bytes as one
    write of everything, at every page size."""
    lens, D, heads = [300, 17, 259], 128, 2
    once, steps = (U.Layout(lens, lens, page, seed=3) for _ in range(2))
    k, v = (U.draw((sum(lens), heads, D), s).to(DEV) for s in (1, 2))
    a, b = (make_cache(once, heads, D, 4, 64, fill=0x11) for _ in range(2))
    B.echo_kv_write(a, once.batch(), k, v)
    first = np.concatenate([[0], np.cumsum(lens)])
    done = [n - 5 for n in lens]
    for step in range(6):
        new = done if step == 0 else [1] * 3
        now = [d + step for d in done]
        rows = np.concatenate([np.arange(first[i] + now[i] - new[i], first[i] + now[i]) for i in range(3)])
        steps.lens = now
        t = torch.from_numpy(rows).to(DEV)
        B.echo_kv_write(b, steps.batch(new=new), k[t], v[t])
    for x, y in zip((a.k_codes, a.v_codes, a.k_params, a.v_params), (b.k_codes, b.v_codes, b.k_params, b.v_params)):
        assert torch.equal(x, y)


def test_strided_rows():
    """Slices of a fused projection, head-major rows and broadcast inputs."""
    heads, D, T = 3, 64, 45
    lay = U.Layout([T], [T], 32)
    fused = U.draw((T, 5, heads, D), 4).to(DEV)
    for k, v in ((fused[:, 1], fused[:, 4]),
                 (fused[:, 0].transpose(0, 1).contiguous().transpose(0, 1), fused[:, 2]),
                 (fused[:, :1, 0].expand(T, heads, D), fused[:1, 3].expand(T, heads, D))):
        cache = make_cache(lay, heads, D, 4, 32, fill=0x5A)
        B.echo_kv_write(cache, lay.batch(), k, v)
        check_written(cache, lay, lay.new, k, v, 0x5A)
    head_major = torch.zeros(heads, T, D, dtype=torch.float32, device=DEV)
    wide = torch.full((T, 2 * heads, D), 3.0, dtype=torch.float32, device=DEV)
    B.echo_kv_read(cache, lay.batch(), head_major.transpose(0, 1), wide[:, heads:])
    want = U.values(*U.quantize(U.host64(v), 4, 32), 32)
    assert np.array_equal(U.host64(wide[:, heads:]), want)
    assert (wide[:, :heads] == 3.0).all()
    assert np.array_equal(U.host64(head_major.transpose(0, 1)), U.values(*U.quantize(U.host64(k), 4, 32), 32))


def test_rows_without_a_place_are_passed_over():
    """Rows behind the last sequence, positions below zero, pages that are no
    pages, positions past the table or past max_len: not written, not read."""
    heads, D = 2, 128
    lay = U.Layout([40, 33, 20, 8], [40, 33, 20, 12], 16, spare=1, seed=1)   # the last brings 12 rows for 8 positions
    lay.table[0, 1] = lay.pages            # one past the last page
    lay.table[1, 0] = -7
    lay.table[2, 1] = 2 ** 31 - 1
    batch = lay.batch(rows=lay.rows + 9, max_len=36)
    k, v = (U.draw((lay.rows + 9, heads, D), s).to(DEV) for s in (1, 2))
    cache = make_cache(lay, heads, D, 4, 128, fill=0x3C)
    B.echo_kv_write(cache, batch, k, v)
    out = [torch.full((lay.rows + 9, heads, D), 9.0, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    B.echo_kv_read(cache, batch, *out)
    rows = U.cache_rows(cache)
    touched = np.zeros((lay.pages, lay.page), bool)
    seen = np.zeros(lay.rows + 9, bool)
    for b in range(4):
        for i in range(lay.new[b]):
            pos = lay.lens[b] - lay.new[b] + i
            page = lay.table[b, pos // 16] if pos >= 0 else -1
            if pos < 0 or pos >= 36 or not 0 <= page < lay.pages:
                continue
            r = lay.start[b] + i
            seen[r] = True
            touched[page, pos % 16] = True
            want = U.quantize(U.host64(k[r]), 4, 128)
            assert np.array_equal(rows[0][0][page, :, pos % 16], want[0])
    assert seen.sum() == (36 - 16) + (33 - 16) + 16 + 8
    for o, x in zip(out, (k, v)):
        want = U.values(*U.quantize(U.host64(x), 4, 128), 128)
        got = o.float().cpu().numpy()
        assert (got[~seen] == 9.0).all()
        assert np.array_equal(got[seen], torch.from_numpy(want[seen]).to(torch.bfloat16).float().numpy())
    raw = cache.v_codes.cpu().numpy().transpose(0, 2, 1, 3)
    assert (raw[~touched] == 0x3C).all()


def test_many_sequences():
    """More sequences than one look-up step covers (64), empty ones among them;
    the rows of one wave belong to many sequences."""
    rng = np.random.default_rng(0)
    new = rng.integers(0, 3, 700).tolist()
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 20, 700))]
    lay = U.Layout(lens, new, 16, seed=8)
    cache = make_cache(lay, 1, 64, 4, 64, fill=0x77)
    k, v = (U.draw((lay.rows, 1, 64), s).to(DEV) for s in (1, 2))
    B.echo_kv_write(cache, lay.batch(), k, v)
    check_written(cache, lay, new, k, v, 0x77)
    out = [torch.zeros(lay.rows, 1, 64, dtype=torch.float32, device=DEV) for _ in "kv"]
    B.echo_kv_read(cache, lay.batch(), *out)
    assert np.array_equal(U.host64(out[0]), U.values(*U.quantize(U.host64(k), 4, 64), 64))


def test_any_index_array_stays_inside():
    """Index arrays of noise: the bytes before and behind every buffer stay as
    they were (the CPU test of the index arithmetic runs the same ranges)."""
    rng = np.random.default_rng(4)
    for trial in range(6):
        seqs, width, rows = 9, 5, 100
        start = rng.integers(-50, 150, seqs + 1).astype(np.int32)
        if trial % 2:
            start = np.sort(start)
        lens = rng.integers(-2 ** 31, 2 ** 31 - 1, seqs).astype(np.int32) if trial < 2 else \
            rng.integers(-20, 120, seqs).astype(np.int32)
        table = rng.integers(-3, 12, (seqs, width)).astype(np.int32)
        batch = B.KVBatch(*(torch.from_numpy(a).to(DEV) for a in (start, lens, table)), rows=rows, max_new=40, max_len=77)
        big = [torch.full((12, 2, 16, n), 0x42, dtype=torch.uint8, device=DEV) for n in (64, 64, 4, 4)]
        part = [t[2:10] for t in big]
        cache = B.KVCache(4, 128, 128, part[0], part[1], part[2].view(torch.int32), part[3].view(torch.int32))
        wide = torch.full((rows + 16, 2, 128), 2.5, dtype=torch.bfloat16, device=DEV)
        B.echo_kv_write(cache, batch, wide[8:-8], wide[8:-8])
        B.echo_kv_read(cache, batch, wide[8:-8], torch.empty_like(wide[8:-8]))
        q = torch.full((rows + 16, 4, 128), 1.0, dtype=torch.bfloat16, device=DEV)
        out = torch.full_like(q, 8.0)
        B.echo_kv_attention(cache, batch, q[8:-8], out[8:-8], 0.1)
        torch.cuda.synchronize()
        for t in big:
            assert (t[:2] == 0x42).all() and (t[10:] == 0x42).all()
        assert (wide[:8] == 2.5).all() and (wide[-8:] == 2.5).all()
        assert (out[:8] == 8.0).all() and (out[-8:] == 8.0).all()


def test_offsets_past_32_bits():
    """A cache of more than 4 GiB of codes: rows in its last pages."""
    heads, D, page = 16, 256, 256
    pages = (1 << 32) // (heads * page * D) + 3
    need = 2 * pages * heads * page * (D + 4 * D // 128)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need + (1 << 30):
        pytest.skip("not enough free device memory")
    cache = B.alloc_kv_cache(pages, page, heads, D, bits=8, group=128, device=DEV)
    n = 2 * page + 7
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device=DEV)
    batch = B.KVBatch(torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                      table, rows=n, max_new=n, max_len=n)
    k, v = (U.draw((n, heads, D), s).to(DEV) for s in (1, 2))
    B.echo_kv_write(cache, batch, k, v)
    out = [torch.zeros(n, heads, D, dtype=torch.float32, device=DEV) for _ in "kv"]
    B.echo_kv_read(cache, batch, *out)
    values = [U.values(*U.quantize(U.host64(x), 8, 128), 128) for x in (k, v)]
    for got, want in zip(out, values):
        assert np.array_equal(U.host64(got), want)
    q = U.draw((n, heads, D), 3).to(DEV)
    o = torch.empty_like(q)
    B.echo_kv_attention(cache, batch, q, o, D ** -0.5)
    i = n - 1
    for h in (0, heads - 1):
        s = values[0][:, h] @ U.host64(q[i, h]) * D ** -0.5
        w = np.exp(s - s.max())
        want = w @ values[1][:, h] / w.sum()
        assert np.abs(U.host64(o[i, h]) - want).max() < 0.01 * np.abs(want).max() + 2 ** -9 * np.abs(want).max()


@pytest.mark.parametrize("bits", [4, 8])
def test_every_step(bits):
    """Every fp16 step: groups whose range is that step's, its midpoint to the
    next and the binary32 neighbours of the midpoint, with elements on and next to
    the codes' midpoints, where a quotient or reciprocal off by one bit shows."""
    top = float(2 ** bits - 1)
    steps = np.arange(0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)
    mid = np.float32((steps + np.append(steps[1:], 65536.0)) / 2 * top)
    low, high = np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(np.inf))
    x = np.zeros((4, len(steps), 64), np.float32)
    x[:, :, 1] = np.stack([np.float32(steps * top), low, mid, high])
    codes = np.arange(20) if bits == 4 else np.r_[0:7, 120:127, 249:255]
    codes = codes[codes < top]
    ties = (codes + 0.5) * steps[:, None]
    for i, t in enumerate((ties.astype(np.float32), np.nextafter(np.float32(ties), np.float32(0)),
                           np.nextafter(np.float32(ties), np.float32(np.inf)))):
        at = 2 + i * len(codes)
        x[:, :, at:at + len(codes)] = np.fmin(t, x[:, :, 1:2])
    rows = x.reshape(-1, 1, 64)
    lay = U.Layout([len(rows)], [len(rows)], 256)
    cache = make_cache(lay, 1, 64, bits, 64)
    k = torch.from_numpy(rows).to(DEV)
    B.echo_kv_write(cache, lay.batch(), k, k)
    torch.cuda.synchronize()
    pages, slots = lay.slots(0, range(len(rows)))
    want = U.quantize(rows.astype(np.float64), bits, 64)
    for stored in U.cache_rows(cache):
        for have, w in zip(stored, want):
            np.testing.assert_array_equal(have[pages, 0, slots], w[:, 0])
