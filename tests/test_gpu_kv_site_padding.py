"""An attention site on a padded batch: rows behind the last sequence bring
nothing into the ranks' messages, whatever earlier calls or the allocator left."""
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


@pytest.mark.parametrize("hidden", [384, 80])              # 80: groups of the message hold elements of two rows
def test_padded_rows_bring_nothing(hidden):
    P, heads, per, D, rows, real = 2, 2, 4, 64, 16, [3, 4]
    cfg = B.make_config()
    lay = U.Layout([9, 20], real, 16)
    weights = [U.draw((heads * per * D, hidden), 5 + p, scale=0.05).to(DEV) for p in range(P)]
    batch = lay.batch(rows=rows)
    a = sim.alloc_attention(P, lay.pages, 16, heads, D, weights, [batch], 4, 64, DEV)
    q, k, v = ([U.draw((rows, h, D), 10 * p + i).to(DEV) for p in range(P)]
               for i, h in enumerate((heads * per, heads, heads)))
    full = lay.batch(new=lay.lens)
    for p in range(P):
        B.echo_kv_write(a.caches[p], full, *(U.draw((sum(lay.lens), heads, D), 50 + i).to(DEV) for i in range(2)))
    r = sim.alloc_ranks(cfg, P, rows * hidden, DEV)
    oS, oL = ([np.zeros(rows * hidden, np.float32) for _ in range(P)] for _ in range(2))
    for left in (float("nan"), 7.0):                       # in the buffers before the call
        for t in a.attended + a.partial:
            t.fill_(left)
        got = sim.attention_site(cfg, r, a, batch, q, k, v, D ** -0.5)
        torch.cuda.synchronize()
        for p in range(P):
            assert (a.partial[p][sum(real):] == 0).all() and a.partial[p].isfinite().all()
            assert a.partial[p][:sum(real)].any(1).all()
        ref, _, _ = O.allreduce(oracle_config(cfg), [host(x.reshape(-1)) for x in a.partial], oS, oL)
        assert_bits_equal(host(got), ref, "output")
        for p in range(P):
            S, L = split_state(r.state[p])
            assert_bits_equal(S, oS[p], "short memory")
            assert_bits_equal(L, oL[p], "long memory")


def test_rows_past_max_new_bring_nothing():
    """Rows that a batch's max_new leaves out count as padding."""
    P, heads, per, D, hidden = 1, 1, 2, 64, 128
    lay = U.Layout([9], [5], 16)
    batch = lay.batch(max_new=3)
    a = sim.alloc_attention(P, lay.pages, 16, heads, D, [U.draw((per * D, hidden), 1).to(DEV)], [batch], 4, 64, DEV)
    a.attended[0].fill_(float("nan"))
    r = sim.alloc_ranks(B.make_config(), P, 5 * hidden, DEV)
    for t in (a.caches[0].k_params, a.caches[0].v_params):
        t.zero_()
    q, k, v = ([U.draw((5, h, D), i).to(DEV)] for i, h in enumerate((per, heads, heads)))
    sim.attention_site(B.make_config(), r, a, batch, q, k, v, 0.1)
    assert (a.partial[0][3:] == 0).all() and a.partial[0][:3].isfinite().all()
