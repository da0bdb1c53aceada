"""Attention over the quantized K/V cache, against the definition in 64 bits on
the cache's own codes.

Tolerance (derived in kv_testutil.attend): half a step of the output type on the
output, 2^-11 of the rounded probabilities' weights, and the binary32 terms."""
import numpy as np
import pytest
import torch

import kv_testutil as U
from error_compensated_bit_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMS = [(bits, D, G) for bits in (4, 8) for D in (64, 128, 256) for G in (32, 64, 128) if G <= D]


class Case:
    """A filled cache, queries, and the 64-bit answer."""

    def __init__(self, lens, new, heads=2, per=4, D=128, bits=4, group=128, page=16, dtype="bf16", seed=0, scale=None,
                 k_scale=1.0, k_offset=0.0, v_scale=1.0, v_offset=0.0, q_scale=1.5, fill=0xFF):
        self.lay = U.Layout(lens, lens, page, seed=seed)
        self.lens, self.new, self.heads, self.per, self.D = lens, new, heads, per, D
        self.bits, self.group, self.dtype = bits, group, dtype
        self.scale = D ** -0.5 if scale is None else scale
        self.cache = B.alloc_kv_cache(self.lay.pages, page, heads, D, bits, group, DEV)
        for t in (self.cache.k_codes, self.cache.v_codes, self.cache.k_params, self.cache.v_params):
            t.view(torch.uint8).fill_(fill)          # unwritten slots: 0xFF parameters are NaN
        rows = sum(lens)
        self.k = U.draw((rows, heads, D), seed + 1, dtype, k_scale, k_offset)
        self.v = U.draw((rows, heads, D), seed + 2, dtype, v_scale, v_offset)
        if rows:
            B.echo_kv_write(self.cache, self.lay.batch(), self.k.to(DEV), self.v.to(DEV))
        self.q = U.draw((sum(new), heads * per, D), seed + 3, dtype, q_scale)

    def batch(self, **kw):
        return self.lay.batch(new=self.new, **kw)

    def run(self, causal=True, window=0, sinks=0, **kw):
        q = self.q.to(DEV)
        out = torch.full_like(q, 33.0)
        B.echo_kv_attention(self.cache, self.batch(**kw), q, out, self.scale, causal, window, sinks)
        torch.cuda.synchronize()
        return out

    def check(self, out, causal=True, window=0, sinks=0):
        eps = torch.finfo(U.DTYPES[self.dtype]).eps
        kq, vq = (U.quantize(U.host64(x), self.bits, self.group) for x in (self.k, self.v))
        k, v = (U.values(*x, self.group) for x in (kq, vq))
        half = 2 ** (self.bits - 1)
        spread = np.abs(vq[0].astype(np.float64) - half) * np.repeat(vq[1], self.group, axis=-1)
        got = U.host64(out)
        assert np.isfinite(got).all()
        first = np.concatenate([[0], np.cumsum(self.lens)])
        at = 0
        for b, (length, n) in enumerate(zip(self.lens, self.new)):
            s = slice(first[b], first[b + 1])
            want, bound = U.attend(U.host64(self.q[at:at + n]), k[s], v[s], length, causal, window, sinks, self.scale,
                                   spread[s])
            off = np.abs(got[at:at + n] - want)
            allowed = bound + eps / 2 * (np.abs(want) + bound) + (2.0 ** -25 if self.dtype == "f16" else 2.0 ** -134)
            assert (off <= allowed).all(), (b, (off / allowed).max(), off.max())
            at += n

    def run_and_check(self, **kw):
        self.check(self.run(**kw), **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bits,D,G", FORMS)
def test_single_tokens_of_every_form(bits, D, G, dtype):
    """One query token per sequence: lengths of one, inside a page, at a tile's
    end, one past it, and several tiles."""
    Case([1, 15, 32, 33, 150], [1] * 5, heads=2, per=3, D=D, bits=bits, group=G, dtype=dtype).run_and_check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bits,D,G", FORMS)
def test_several_tokens_of_every_form(bits, D, G, dtype):
    """Ragged rows of 1 to 45 new tokens with and without earlier positions: more
    than 64 and more than 128 rows of one K/V head."""
    Case([45, 70, 1, 9], [45, 33, 1, 0], heads=2, per=4, D=D, bits=bits, group=G, dtype=dtype, seed=1).run_and_check()


@pytest.mark.parametrize("per", [1, 2, 3, 5, 8, 16, 17, 40])
@pytest.mark.parametrize("new", [1, 2, 5])
def test_heads_per_kv_head(per, new):
    """Every tile count of a wave (16, 32, 64 rows) and rows that end inside a tile."""
    Case([77, 20], [new, new], heads=3, per=per, D=64, group=64, seed=per).run_and_check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(page):
    Case([300, 31], [2, 31], page=page, D=128, group=64, seed=page).run_and_check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (32, 4), (33, 40), (64, 0), (100, 3), (1000, 4)])
@pytest.mark.parametrize("new", [1, 20])
def test_window_and_first_tokens(window, sinks, new):
    Case([310, 130, 40], [new, new, new], heads=1, per=4, D=64, group=32, seed=window).run_and_check(
        window=window, sinks=sinks)


def test_not_causal():
    Case([130, 20, 5], [9, 20, 5], seed=3).run_and_check(causal=False)
    Case([260, 3], [1, 3], seed=4, D=64, group=64, dtype="f16").run_and_check(causal=False)


def test_rows_that_see_nothing_become_zero():
    """Sequences without keys, rows before the first position, pages that are no
    pages: exact zeros; the other rows as ever; rows behind the last sequence untouched."""
    c = Case([50, 0, 3], [2, 4, 5], seed=5, fill=0xFF)       # 4 rows and no keys; 5 rows for 3 positions
    batch = c.batch(rows=11 + 3, max_len=50)
    q = torch.cat([c.q, c.q[:3]]).to(DEV)
    out = torch.full_like(q, 33.0)
    B.echo_kv_attention(c.cache, batch, q, out, c.scale)
    assert (out[2:6] == 0).all() and (out[6:8] == 0).all() and (out[11:] == 33.0).all()
    c.lens, c.new, keep = [50, 3], [2, 3], c.q
    c.q = torch.cat([keep[:2], keep[8:]])
    c.check(torch.cat([out[:2], out[8:11]]))
    batch.page_table.fill_(c.lay.pages)          # a table that names no page
    out = torch.full_like(q, 33.0)
    B.echo_kv_attention(c.cache, batch, q, out, c.scale)
    assert (out[:11] == 0).all() and (out[11:] == 33.0).all()


def test_the_widest_window_with_rows_before_the_first_position():
    """A window of 2^31 - 1 hides nothing, also beside rows whose position is negative."""
    c = Case([40], [60], seed=28)
    want = c.run()
    assert torch.equal(c.run(window=2 ** 31 - 1), want) and (want[:20] == 0).all()
    assert torch.equal(c.run(window=2 ** 31 - 1, sinks=2 ** 31 - 1), want)
    c.new, c.q = [40], c.q[20:]
    c.check(want[20:])


def test_a_page_that_is_none_hides_its_keys():
    c = Case([100], [1], page=16, seed=6)
    batch = c.batch()
    batch.page_table[0, 2] = -1
    q = c.q.to(DEV)
    out = torch.empty_like(q)
    B.echo_kv_attention(c.cache, batch, q, out, c.scale)
    hide = np.r_[0:32, 48:100]
    k, v = (U.values(*U.quantize(U.host64(x), 4, 128), 128)[hide] for x in (c.k, c.v))
    for h in range(8):
        s = k[:, h // 4] @ U.host64(c.q[0, h]) * c.scale
        w = np.exp(s - s.max())
        want = w @ v[:, h // 4] / w.sum()
        assert np.abs(U.host64(out[0, h]) - want).max() <= 2.0 ** -8 * np.abs(want).max() + 2.0 ** -10


@pytest.mark.parametrize("new", [1, 30, 300])
def test_long_keys_are_split_and_joined(new):
    """Few rows and many keys: parts of the keys in different blocks, one
    sequence short enough to be whole."""
    c = Case([5000, 60, 2500], [new, min(new, 60), new], heads=1, per=1, D=64, group=64, page=64, seed=new)
    assert B.echo_kv_workspace_bytes(c.cache, c.batch(), 1) > 0
    c.run_and_check()
    c.run_and_check(window=2000, sinks=5)


def test_distributions():
    """Peaked and flat softmaxes, steps from subnormal to huge, one-sided values,
    constant groups, large and tiny queries."""
    Case([200], [3], q_scale=40.0, seed=1).run_and_check()                       # one key takes all
    Case([200], [3], q_scale=1e-3, seed=2).run_and_check()                       # all keys alike
    Case([200], [3], q_scale=1e-30, k_scale=1e3, seed=3).run_and_check()
    Case([200], [3], q_scale=1e20, k_scale=1e-3, scale=1e-18, seed=4).run_and_check()
    Case([200], [3], v_scale=1e-5, seed=5, dtype="f16").run_and_check()          # subnormal steps
    Case([200], [3], v_scale=3000.0, seed=6).run_and_check()
    Case([200], [3], v_offset=100.0, seed=7).run_and_check()
    Case([200], [3], k_offset=30.0, seed=8).run_and_check()
    Case([200], [3], v_scale=0.0, v_offset=2.0, k_scale=0.0, seed=9).run_and_check()   # constant groups
    Case([200], [3], scale=0.0, seed=10).run_and_check()
    Case([200], [3], scale=-0.3, seed=11).run_and_check()
    Case([200], [3], bits=8, v_scale=1e4, q_scale=8.0, dtype="f16", seed=12).run_and_check()


def test_steps_that_grow_along_the_keys():
    """Value steps that grow by 2^20 over the sequence (the normaliser has to
    move) and scores that grow (the running maximum has to)."""
    c = Case([256], [1], heads=1, per=4, seed=20)
    grow = torch.exp2(torch.linspace(-12, 8, 256))[:, None, None]
    c.v = (c.v.float() * grow).to(torch.bfloat16)
    c.k = (c.k.float() * torch.linspace(0.05, 6, 256)[:, None, None]).to(torch.bfloat16)
    for order in (slice(None), slice(None, None, -1)):
        c.k, c.v = c.k[list(range(256))[order]], c.v[list(range(256))[order]]
        B.echo_kv_write(c.cache, c.lay.batch(), c.k.to(DEV), c.v.to(DEV))
        c.run_and_check()


def test_zero_query_rows_average_the_values():
    c = Case([90], [4], seed=21)
    c.q[1] = 0
    c.run_and_check()


def test_strided_queries_and_outputs():
    c = Case([64, 20], [5, 3], heads=2, per=3, D=64, group=64, seed=22)
    fused = torch.zeros(8, 4, 6, 64, dtype=torch.bfloat16, device=DEV)
    fused[:, 2] = c.q.to(DEV)
    fused[:, 3] = 5.0
    B.echo_kv_attention(c.cache, c.batch(), fused[:, 2], fused[:, 1], c.scale)
    c.check(fused[:, 1])
    assert (fused[:, 3] == 5.0).all() and (fused[:, 0] == 0).all()
    major = torch.zeros(6, 8, 64, dtype=torch.bfloat16, device=DEV)
    q_major = c.q.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    B.echo_kv_attention(c.cache, c.batch(), q_major, major.transpose(0, 1), c.scale)
    c.check(major.transpose(0, 1))


def test_bounds_larger_than_needed():
    """max_new and max_len are bounds: larger ones give the same outputs up to
    the split's rounding."""
    c = Case([64, 20], [5, 3], seed=23)
    c.check(c.run(max_new=200, max_len=40000))
    c.check(c.run(max_new=8, max_len=64))


def test_rows_past_max_new_are_not_computed():
    c = Case([64], [9], seed=24)
    out = c.run(max_new=4)
    assert (out[4:] == 33.0).all()
    whole = c.run()
    assert torch.equal(out[:4], whole[:4])


def test_repeats_give_the_same_bits():
    c = Case([3000, 40], [2, 2], heads=1, per=4, seed=25)
    a = c.run()
    for _ in range(3):
        assert torch.equal(a, c.run())


def test_other_streams():
    """Calls on a side stream, by object and by handle, and with the side stream
    current; two at once on two streams, each with its own workspace."""
    c = Case([3000], [1], heads=1, per=4, seed=26)
    want = c.run()
    q, st = c.q.to(DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (st, st.cuda_stream):
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        B.echo_kv_attention(c.cache, c.batch(), q, out, c.scale, stream=stream)
        st.synchronize()
        assert torch.equal(out, want)
    batch, outs, streams = c.batch(), [torch.zeros_like(q) for _ in range(2)], [st, torch.cuda.Stream()]
    calls = [B.prepare_kv_attention(c.cache, batch, q, o, c.scale, stream=s) for o, s in zip(outs, streams)]
    torch.cuda.synchronize()
    for _ in range(20):
        for call in calls:
            call()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_step_captured_and_replayed():
    """Write, attention (split and joined) and read captured together; each
    replay, with new rows and a new length in the same buffers, equals the eager calls."""
    lens, heads, D = [2100, 900], 2, 128
    lay = U.Layout([n + 8 for n in lens], [1, 1], 64, seed=2)
    caches = [B.alloc_kv_cache(lay.pages, 64, heads, D, device=DEV) for _ in range(2)]
    lay.lens = list(lens)
    full = lay.batch(new=lens)
    k0, v0 = (U.draw((sum(lens), heads, D), s).to(DEV) for s in (1, 2))
    for c in caches:
        c.k_codes.zero_()                       # the whole array is compared
        B.echo_kv_write(c, full, k0, v0)
    batch = lay.batch(new=[1, 1], max_len=2200)
    k, v = (torch.zeros(2, heads, D, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    q = torch.zeros(2, 8, D, dtype=torch.bfloat16, device=DEV)
    out, eager = torch.zeros_like(q), torch.zeros_like(q)
    back = [torch.zeros_like(k) for _ in "kv"]
    assert B.echo_kv_workspace_bytes(caches[0], batch, 8) > 0
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.echo_kv_write(caches[0], batch, k, v)
        B.echo_kv_attention(caches[0], batch, q, out, D ** -0.5)
        B.echo_kv_read(caches[0], batch, *back)
    for step in range(4):
        batch.kv_len.copy_(torch.tensor([n + step + 1 for n in lens], dtype=torch.int32))
        for t, s in ((k, 10), (v, 20), (q, 30)):
            t.copy_(U.draw(tuple(t.shape), s + step))
        g.replay()
        noise = torch.randn(1 << 18, device=DEV).square()
        B.echo_kv_write(caches[1], batch, k, v)
        B.echo_kv_attention(caches[1], batch, q, eager, D ** -0.5)
        torch.cuda.synchronize()
        assert noise.isfinite().all()
        assert torch.equal(out, eager)
        same = torch.equal(caches[0].k_codes, caches[1].k_codes)
        assert same
        want = U.values(*U.quantize(U.host64(k), 4, 128), 128)
        assert torch.equal(back[0].cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_two_graphs_with_their_own_workspaces():
    c = Case([3000], [1], heads=1, per=4, seed=27)
    want = c.run()
    q, batch = c.q.to(DEV), c.batch()
    graphs, outs, keep = [], [], []
    for _ in range(2):
        o, g = torch.zeros_like(q), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            call = B.prepare_kv_attention(c.cache, batch, q, o, c.scale, stream=torch.cuda.current_stream())
            call()
        graphs.append(g), outs.append(o), keep.append(call)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, want)


@pytest.mark.parametrize("seqs,per,new,D,bits,group", [
    (270, 4, 1, 128, 4, 128), (270, 8, 1, 64, 8, 32), (270, 3, 1, 256, 8, 64),     # one tile of rows, 4 waves
    (140, 6, 4, 128, 4, 64), (20, 6, 4, 128, 4, 64),                               # 24 rows, many and few pairs
    (140, 5, 8, 256, 4, 128), (140, 7, 8, 256, 8, 32), (20, 10, 10, 256, 4, 64),   # 256 elements, 40, 56 and 100 rows
    (20, 10, 4, 64, 8, 32), (20, 10, 4, 128, 8, 32),                               # 40 rows, few pairs
    (140, 13, 8, 64, 4, 64), (140, 13, 8, 128, 8, 128), (5, 43, 3, 64, 8, 64),     # 104 and 129 rows
])
def test_forms_chosen_by_pairs_and_rows(seqs, per, new, D, bits, group):
    """Sizes on both sides of every choice of kernel form, with sequences of very
    different lengths in one call."""
    lens = np.random.default_rng(seqs + per).integers(1, 45, seqs).tolist()
    lens[seqs // 2] = 333
    Case(lens, [min(new, n) for n in lens], heads=1, per=per, D=D, bits=bits, group=group, seed=30).run_and_check()


@pytest.mark.parametrize("D,new", [(64, 300), (128, 300), (256, 150), (128, 40), (64, 120)])
def test_many_rows_split_and_joined(D, new):
    c = Case([4200, 170], [new, 60], heads=1, per=1, D=D, group=64, page=64, seed=31)
    assert B.echo_kv_workspace_bytes(c.cache, c.batch(), 1) > 0
    c.run_and_check()


def test_one_workspace_for_calls_that_follow_each_other():
    """A workspace of the largest call serves smaller ones in between; a call
    leaves its counters at 0; one that is too small is refused."""
    cases = [Case([4000, 700], [3, 1], heads=1, per=4, seed=32), Case([2500], [1], heads=2, per=2, D=64, group=64, seed=33),
             Case([6000, 3, 1200], [40, 3, 40], heads=1, per=8, seed=34)]
    sizes = [B.echo_kv_workspace_bytes(c.cache, c.batch(), c.heads * c.per) for c in cases]
    assert min(sizes) > 0 and len(set(sizes)) == 3
    want = [c.run() for c in cases]
    work = torch.zeros(max(sizes), dtype=torch.uint8, device=DEV)
    for i in (0, 1, 2, 1, 0, 2):
        c = cases[i]
        q = c.q.to(DEV)
        out = torch.zeros_like(q)
        B.echo_kv_attention(c.cache, c.batch(), q, out, c.scale, workspace=work)
        assert torch.equal(out, want[i])
        assert not work[:1024].any()
        with pytest.raises(B.EchoError):
            B.echo_kv_attention(c.cache, c.batch(), q, out, c.scale, workspace=work[:sizes[i] - 4])


def test_empty_calls_and_sequences():
    """No sequences, no rows, sequences without rows or without keys: nothing but the given rows is written."""
    c = Case([50, 0, 7, 20], [4, 0, 0, 1], seed=35)
    c.run_and_check()
    q = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device=DEV)
    none = B.KVBatch(torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV),
                     torch.zeros(0, 4, dtype=torch.int32, device=DEV), 0, 0, 0)
    B.echo_kv_attention(c.cache, none, q, torch.empty_like(q), 0.1)
    torch.cuda.synchronize()
