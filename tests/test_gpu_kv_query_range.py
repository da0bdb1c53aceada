"""Queries of one call whose sizes differ by many powers of two, scales at the
ends of binary32, and queries that are no numbers: no row's query changes
another row's result.

Bound: kv_attend64.attend_at's.  An element of a query enters the products with
an error of 2^-25 of its row's largest element at most, a score with 2^-25 max|q|
sum_d |c_d s|.  For drawn rows (max|q| about 4.5, c s about 5 at most, mean |k|
|q| about 1) that is 23 D 2^-25, a twelfth of the D (D + 8) 2^-23 that the bound's
first term allows at 64 elements, less above."""
import numpy as np
import pytest
import torch

import kv_testutil as U
from error_compensated_bit_amd import binding as B
from kv_attend64 import Sequences

pytestmark = pytest.mark.gpu
FORMS = [(128, 4, 128), (64, 4, 32), (256, 4, 128), (128, 8, 64), (64, 8, 64), (256, 8, 32)]


def run(s, q, n, scale=None, **mask):
    q = q.to(s.device)
    out = torch.full_like(q, 33.0)
    B.echo_kv_attention(s.cache, s.batch([n], s.lens), q, out, s.scale if scale is None else scale, **mask)
    torch.cuda.synchronize()
    return out


def filled(n, D=128, bits=4, group=128, dtype="bf16", seed=0, length=150, **kw):
    s = Sequences([length], D=D, bits=bits, group=group, dtype=dtype, seed=seed, **kw)
    s.write([(0, length)])
    return s, s.queries(n)


def check(s, out, q, n, rows=None, **kw):
    rows = np.arange(n) if rows is None else np.asarray(rows)
    s.check(out[rows], q[rows], 0, s.lens[0] - n + rows, s.lens[0], **kw)


@pytest.mark.parametrize("far", [12, 20, 30, 60, 100])
@pytest.mark.parametrize("n", [3, 40])                       # few rows of a K/V head, many
@pytest.mark.parametrize("D,bits,group", FORMS)
def test_rows_of_very_different_size(D, bits, group, n, far):
    """One token, then one head, 2^far times larger than the others: those keep their bits."""
    for what in ("token", "head", "small"):
        s, q = filled(n, D, bits, group, seed=far)
        if what == "token":
            q[1] *= 2.0 ** far
        elif what == "head":
            q[:, 2] *= 2.0 ** far
        else:
            q[1:] *= 2.0 ** -far
        check(s, run(s, q, n), q, n)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("D,bits,group", FORMS)
def test_half_precision_rows_of_very_different_size(D, bits, group, n):
    s, q = filled(n, D, bits, group, dtype="f16", seed=1)
    q[1] *= 2.0 ** 13
    q[2] *= 2.0 ** -13
    check(s, run(s, q, n), q, n)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("top", [2.0 ** 119, 2.0 ** 123, 2.0 ** 126, 2.0 ** 127])
def test_the_largest_queries_leave_the_other_rows(n, top):
    """A row near the end of bf16's range whose own scores fit binary32 (a single large element)."""
    s, q = filled(n, seed=2)
    q[1] = 0
    q[1, :, 5] = top
    out = run(s, q, n)
    check(s, out, q, n, [i for i in range(n) if i != 1])
    assert out[1].isfinite().all()


@pytest.mark.parametrize("n", [3, 40])
def test_all_rows_near_the_end_of_the_range(n):
    """One key holds all the weight; its values come back."""
    s, q = filled(n, seed=3)
    q[:] = 0
    q[:, :, 5] = 2.0 ** 126
    out = U.host64(run(s, q, n))
    k, v = (U.values(*U.quantize(U.host64(x), 4, 128), 128) for x in s.kv[0])
    for i in range(n):
        for h in range(s.heads * s.per):
            want = v[np.argmax(k[:150 - n + i + 1, h // s.per, 5]), h // s.per]
            # one probability and its product with the step round to f16, the output to bf16
            assert (np.abs(out[i, h] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * np.abs(v).max()).all()


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("far", range(16, 44))
def test_scores_of_every_size(n, far):
    """Scores whose binary32 neighbours lie further apart than a probability may
    exceed the running maximum: results stay finite."""
    s, q = filled(n, seed=far)
    q *= 2.0 ** far
    check(s, run(s, q, n), q, n)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_the_largest_scales(n, sign):
    """Scales up to the largest binary32 number, beyond which log2(e) would take them."""
    s, q = filled(n, seed=4)
    for scale in (1e38, 3e38, 3.4028234e38):
        small = (q.float() / 3e38 * 8).to(torch.bfloat16)
        check(s, run(s, small, n, scale=sign * scale), small, n, scale=sign * scale)


@pytest.mark.parametrize("n", [3, 40])
def test_scale_zero_weighs_every_key_the_same(n):
    """... also for queries of 2^100 and more."""
    s, q = filled(n, seed=5)
    q = (q.float() * 2.0 ** 100).to(torch.bfloat16)
    check(s, run(s, q, n, scale=0.0), q, n, scale=0.0)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D,bits,group", [(128, 4, 128), (64, 8, 32), (256, 4, 64)])
def test_rows_that_are_no_numbers(D, bits, group, bad, n):
    """A NaN or infinite element makes its own row NaN and no other.  The others
    are right within the bound, not bit for bit: a row whose maximum is not
    settled lets its whole wave's maxima rise, and a probability rounds to f16
    relative to its row's."""
    s, q = filled(n, D, bits, group, seed=6)
    s.kv[0][0] = s.kv[0][0].abs() + 1.0                 # keys whose products with an infinity have one sign
    s.write([(0, 150)])
    q[1, 3, 7] = bad
    out = run(s, q, n)
    assert out[1, 3].isnan().all()
    q[1, 3] = 0
    clean = run(s, q, n)
    check(s, clean, q, n)
    out[1, 3] = clean[1, 3]
    check(s, out, q, n)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("D,bits,group", [(128, 4, 128), (64, 8, 32), (256, 4, 64)])
def test_a_row_whose_scores_are_all_minus_infinity(D, bits, group, n):
    """Infinity less infinity in the softmax: NaN, not the 0 of a row that sees nothing."""
    s, q = filled(n, D, bits, group, seed=6)
    s.kv[0][0] = s.kv[0][0].abs() + 1.0
    s.kv[0][0][:, :, 7] += 2.0                          # no key's code is 0 there
    s.write([(0, 150)])
    codes, _, _ = U.quantize(U.host64(s.kv[0][0]), bits, group)
    assert (codes[:, :, 7] > 0).all()
    q[1, 3, 7] = -float("inf")
    out = run(s, q, n)
    assert out[1, 3].isnan().all()
    q[1, 3] = 0
    out[1, 3] = run(s, q, n)[1, 3]
    check(s, out, q, n)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_no_numbers_and_see_nothing(bad):
    s, q = filled(3, seed=7)
    q[:] = bad
    out = torch.full_like(q, 33.0).to(s.device)
    B.echo_kv_attention(s.cache, s.batch([3], [0], max_len=64), q.to(s.device), out, s.scale)
    assert (out == 0).all()
