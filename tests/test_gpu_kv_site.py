"""A tensor-parallel attention site as a serving loop runs it: prompts, then
tokens one by one, each through write, attention, output projection and the
all-reduce of the ranks' partial products.

Every stage is checked on what the stage before it gave: the cache's codes
against the quantizer's definition bit for bit, attention against 64 bits on
those codes within kv_testutil's bound, the projection within half a bf16 step
and the binary32 sums, the all-reduce and its error state against the CPU
oracle bit for bit."""
import numpy as np
import pytest
import torch

import kv_testutil as U
import oracle as O
from echo_testutil import assert_bits_equal, host, oracle_config, split_state
from error_compensated_bit_amd import binding as B
from error_compensated_bit_amd import sim

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("P,heads,per,D,bits,group", [(2, 2, 4, 64, 4, 64), (4, 1, 6, 128, 8, 128)])
def test_prompts_then_tokens(P, heads, per, D, bits, group):
    hidden, page = 384, 16
    prompts, steps = [37, 1, 64], 4
    cfg = B.make_config()
    weights = [U.draw((heads * per * D, hidden), 90 + p, scale=0.05) for p in range(P)]
    # sequences of one page table over the whole run
    lay = U.Layout([n + steps for n in prompts], prompts, page)
    table = torch.from_numpy(lay.table).to(DEV)

    def batch(new, lens):
        start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        return B.KVBatch(start, torch.tensor(lens, dtype=torch.int32, device=DEV), table, sum(new), max(new), max(lens))

    calls = [(prompts, prompts)] + [([1] * len(prompts), [n + 1 + s for n in prompts]) for s in range(steps)]
    batches = [batch(*c) for c in calls]
    a = sim.alloc_attention(P, lay.pages, page, heads, D, [w.to(DEV) for w in weights], batches, bits, group, DEV)
    seen = [[np.zeros((0, heads, D))] * len(prompts) for _ in range(2 * P)]     # every key and value so far
    for step, ((new, lens), b) in enumerate(zip(calls, batches)):
        rows = sum(new)
        q, k, v = ([U.draw((rows, h, D), 1000 * step + 10 * p + i, scale=1.2) for p in range(P)]
                   for i, h in enumerate((heads * per, heads, heads)))
        r = sim.alloc_ranks(cfg, P, rows * hidden, DEV)
        got = sim.attention_site(cfg, r, a, b, *([t.to(DEV) for t in x] for x in (q, k, v)), D ** -0.5)
        torch.cuda.synchronize()
        partial = [a.partial[p][:rows] for p in range(P)]
        for p in range(P):
            stored = U.cache_rows(a.caches[p])
            att = U.host64(a.attended[p][:rows])
            at = 0
            for s, (n, length) in enumerate(zip(new, lens)):
                kv = []
                for i, x in enumerate((k, v)):
                    seen[2 * p + i][s] = np.concatenate([seen[2 * p + i][s], U.host64(x[p][at:at + n])])
                    code, sc, zero = U.quantize(seen[2 * p + i][s], bits, group)
                    pages, slots = lay.slots(s, range(length))
                    for have, want in zip(stored[i], (code, sc, zero)):
                        np.testing.assert_array_equal(have[pages, :, slots], want)
                    kv.append((U.values(code, sc, zero, group), code, sc))
                spread = np.abs(kv[1][1].astype(np.float64) - 2 ** (bits - 1)) * np.repeat(kv[1][2], group, axis=-1)
                want, bound = U.attend(U.host64(q[p][at:at + n]), kv[0][0], kv[1][0], length, True, 0, 0, D ** -0.5,
                                       spread)
                err = np.abs(att[at:at + n] - want)
                assert (err <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all(), (step, p, s, err.max())
                at += n
            w = U.host64(weights[p])
            x = att.reshape(rows, -1)
            want = x @ w
            sums = x.shape[1] * 2.0 ** -23 * (np.abs(x) @ np.abs(w))     # as many roundings as terms, any order
            assert (np.abs(U.host64(partial[p]) - want) <= sums + 2.0 ** -8 * (np.abs(want) + sums)).all()
        oS, oL = ([np.zeros(rows * hidden, np.float32) for _ in range(P)] for _ in range(2))
        ref, _, _ = O.allreduce(oracle_config(cfg), [host(y.reshape(-1)) for y in partial], oS, oL)
        assert_bits_equal(host(got), ref, f"step {step} output")
        for p in range(P):
            S, L = split_state(r.state[p])
            assert_bits_equal(S, oS[p], f"step {step} rank {p} short memory")
            assert_bits_equal(L, oL[p], f"step {step} rank {p} long memory")
    assert not a.workspace[:4 * 256].any()       # arrival counters are back at 0
