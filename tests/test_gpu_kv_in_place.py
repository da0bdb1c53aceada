"""Attention whose outputs take the queries' place, in every way that a call is
cut into blocks: the bits of a call with an array of its own."""
import pytest
import torch

from error_compensated_bit_amd import binding as B
from kv_attend64 import Sequences

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("uneven", [False, True])
@pytest.mark.parametrize("lens,new,heads,per,split", [
    ([150, 40], [3, 1], 2, 4, False),          # few rows
    ([150, 90], [70, 40], 2, 4, False),        # many, several blocks of rows
    ([6000, 700], [2, 1], 1, 4, True),         # few, split keys
    ([5000, 300], [200, 200], 1, 2, True),     # many, split keys
])
def test_outputs_in_the_queries_place(lens, new, heads, per, split, uneven):
    s = Sequences(lens, heads=heads, per=per, page=64, seed=len(lens))
    s.write([(0, n) for n in lens])
    q = s.queries(sum(new))
    if uneven:
        q[::3] *= 2.0 ** 20
    q = q.to(s.device)
    batch = s.batch(new, lens)
    assert (B.echo_kv_workspace_bytes(s.cache, batch, heads * per) > 0) == split
    want = torch.empty_like(q)
    B.echo_kv_attention(s.cache, batch, q, want, s.scale)
    for _ in range(5):
        both = q.clone()
        B.echo_kv_attention(s.cache, batch, both, both, s.scale)
        assert torch.equal(both, want)
