"""The position of a query row is kv_len - n + i, whatever the call's bounds
are: keys from max_len on or past the page table are not there, but the rows
stay where the write puts them."""
import numpy as np
import pytest
import torch

from error_compensated_bit_amd import binding as B
from kv_attend64 import Sequences

pytestmark = pytest.mark.gpu
MASKS = [dict(), dict(window=9), dict(window=20, sinks=3), dict(causal=False)]


def attend(s, q, batch, **mask):
    q = q.to(s.device)
    out = torch.full_like(q, 33.0)
    B.echo_kv_attention(s.cache, batch, q, out, s.scale, **mask)
    torch.cuda.synchronize()
    return out


def check(s, out, q, new, lens, keys, **mask):
    at = 0
    for b, (n, length) in enumerate(zip(new, lens)):
        s.check(out[at:at + n], q[at:at + n], b, np.arange(length - n, length), keys[b], **mask)
        at += n


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("new", [[4, 3], [40, 37]])        # few rows of a K/V head, many
@pytest.mark.parametrize("D,bits,group", [(128, 4, 128), (64, 8, 32), (256, 4, 64)])
def test_lengths_past_max_len(D, bits, group, new, mask):
    s = Sequences([64, 41], D=D, bits=bits, group=group)
    s.write([(0, 64), (0, 41)])
    q = s.queries(sum(new))
    lens = [66, 41]
    out = attend(s, q, s.batch(new, lens, max_len=64), **mask)
    check(s, out, q, new, lens, [64, 41], **mask)


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("new", [[4, 3], [40, 37]])
def test_lengths_past_the_page_table(new, mask):
    """A table one page too narrow."""
    s = Sequences([80, 41], seed=1)
    s.write([(0, 80), (0, 41)])
    q = s.queries(sum(new))
    out = attend(s, q, s.batch(new, [79, 41], table=s.lay.table[:, :4]), **mask)
    check(s, out, q, new, [79, 41], [64, 41], **mask)


@pytest.mark.parametrize("length", [65, 100, 2000, 2 ** 30 + 7, 2 ** 31 - 1])
@pytest.mark.parametrize("n", [3, 40])
def test_rows_far_behind_the_keys(n, length):
    """Every key, the first ones only, or nothing is left of what such rows see."""
    s = Sequences([64], seed=2)
    s.write([(0, 64)])
    q = s.queries(n)
    for mask in (dict(), dict(window=30), dict(window=30, sinks=5), dict(window=60, sinks=40),
                 dict(window=2 ** 31 - 1), dict(causal=False)):
        out = attend(s, q, s.batch([n], [length], max_len=64), **mask)
        s.check(out, q, 0, np.arange(length - n, length), 64, **mask)


@pytest.mark.parametrize("length", [-1, -5, -2 ** 31])
def test_lengths_below_zero_see_nothing(length):
    s = Sequences([64], seed=3)
    s.write([(0, 64)])
    q = s.queries(5)
    for mask in MASKS:
        assert (attend(s, q, s.batch([5], [length], max_len=64), **mask) == 0).all()


@pytest.mark.parametrize("mask", MASKS)
def test_rows_behind_the_packed_arrays(mask):
    """The last sequence names more rows than the arrays have: those there keep
    the positions that the write gives them."""
    s = Sequences([50, 40], seed=4)
    s.write([(0, 50), (0, 40)])
    batch = s.batch([4, 6], [50, 40], rows=7, max_new=6)
    q = s.queries(7)
    out = attend(s, q, batch, **mask)
    s.check(out[:4], q[:4], 0, np.arange(46, 50), 50, **mask)
    s.check(out[4:], q[4:], 1, np.arange(34, 37), 40, **mask)


def test_split_keys_past_max_len():
    """Few rows, keys in several blocks."""
    s = Sequences([4100], heads=1, per=4, D=64, group=64, page=64, seed=5)
    s.write([(0, 4100)])
    q = s.queries(3)
    batch = s.batch([3], [4105], max_len=4100)
    assert B.echo_kv_workspace_bytes(s.cache, batch, 4) > 0
    for mask in (dict(), dict(window=2500, sinks=40)):
        s.check(attend(s, q, batch, **mask), q, 0, np.arange(4102, 4105), 4100, **mask)


def test_a_step_writes_and_attends_at_the_same_positions():
    """A step whose lengths have outgrown max_len: rows that still have a place
    see their own new key."""
    s = Sequences([64], heads=1, per=1, seed=6)
    s.write([(0, 62)])
    batch = s.batch([4], [66], max_len=64)              # positions 62 .. 65; 64 and 65 have no place
    k, v = (torch.cat([t[62:], t[:2]]).to(s.device) for t in s.kv[0])
    B.echo_kv_write(s.cache, batch, k, v)
    q = s.queries(4)
    s.check(attend(s, q, batch, window=1), q, 0, np.arange(62, 66), 64, window=1)
