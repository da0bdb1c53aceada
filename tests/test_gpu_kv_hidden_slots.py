"""Slots that no row sees may hold anything: only the positions that a window
and the first keys leave visible are written, all others keep bytes that read
as NaN or as a step near the largest."""
import numpy as np
import pytest
import torch

from error_compensated_bit_amd import binding as B
from kv_attend64 import Sequences

pytestmark = pytest.mark.gpu
FILLS = [0xFF, 0x7B]          # parameters: NaN; steps and zeros of 61280, 2^27 times the steps of the values here


def run(s, q, batch, **mask):
    q = q.to(s.device)
    out = torch.full_like(q, 33.0)
    B.echo_kv_attention(s.cache, batch, q, out, s.scale, **mask)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("window,sinks", [(50, 0), (50, 3), (33, 37), (1, 1), (1, 0)])
@pytest.mark.parametrize("new", [1, 5, 40])                # 40 new rows: many rows of a K/V head
@pytest.mark.parametrize("D,bits,group,page", [(128, 4, 128, 16), (64, 8, 32, 64), (256, 4, 64, 32), (128, 8, 32, 256)])
def test_only_visible_positions_are_written(D, bits, group, page, new, window, sinks, fill):
    lens = [301, 150]
    s = Sequences(lens, D=D, bits=bits, group=group, page=page, fill=fill, seed=window, v_scale=2.0 ** -8)
    if sinks:
        s.write([(0, sinks)] * 2)
    s.write([(n - new - window + 1, n) for n in lens])
    q = s.queries(2 * new)
    out = run(s, q, s.batch([new] * 2, lens), window=window, sinks=sinks)
    for b, n in enumerate(lens):
        rows = slice(b * new, (b + 1) * new)
        s.check(out[rows], q[rows], b, np.arange(n - new, n), n, window=window, sinks=sinks)


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("computed", [4, 40])
def test_positions_behind_the_computed_rows(computed, fill):
    """max_new cuts a sequence's rows: the positions of the others need no contents."""
    n = computed + 7
    s = Sequences([90], fill=fill, seed=1, v_scale=2.0 ** -8)
    s.write([(0, 90 - 7)])
    q = s.queries(n)
    out = run(s, q, s.batch([n], [90], max_new=computed))
    s.check(out[:computed], q[:computed], 0, np.arange(90 - n, 90 - 7), 90)
    assert (out[computed:] == 33.0).all()


@pytest.mark.parametrize("fill", FILLS)
def test_split_keys(fill):
    """The window's first tile and the first keys' last one lie in different blocks."""
    s = Sequences([6000], heads=1, per=4, D=64, group=64, page=64, fill=fill, seed=2, v_scale=2.0 ** -8)
    s.write([(0, 5)])
    s.write([(6000 - 4999, 6000)])
    q = s.queries(1)
    batch = s.batch([1], [6000])
    assert B.echo_kv_workspace_bytes(s.cache, batch, 4, window=4999, sinks=5) > 0
    s.check(run(s, q, batch, window=4999, sinks=5), q, 0, [5999], 6000, window=4999, sinks=5)
