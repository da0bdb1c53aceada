"""An attention site on a padded batch, without a GPU: rows that the attention
leaves as they were are zeros in what the projection multiplies."""
import torch

from error_compensated_bit_amd import binding as B
from error_compensated_bit_amd import sim


def test_rows_that_attention_leaves_are_zeros(monkeypatch):
    rows, real, hidden, heads, D = 6, 4, 32, 2, 64

    def attention(cache, batch, q, out, scale, **kw):
        out[:real] = 1.0

    monkeypatch.setattr(B, "echo_kv_write", lambda *a, **kw: None)
    monkeypatch.setattr(B, "echo_kv_attention", attention)
    monkeypatch.setattr(sim, "allreduce", lambda cfg, r, xs, stream=None: xs)
    weights = [torch.ones(heads * D, hidden) for _ in range(2)]
    a = sim.AttentionRanks([None, None], weights, None, [torch.full((rows + 2, heads, D), float("nan")) for _ in range(2)],
                           [torch.full((rows + 2, hidden), float("nan")) for _ in range(2)])
    r = sim.Ranks(2, rows * hidden, [], [], [], None)
    x = [torch.zeros(rows, heads, D)] * 2
    for part in sim.attention_site(None, r, a, B.KVBatch(None, None, None, rows, rows, rows), x, x, x, 0.1):
        part = part.reshape(rows, hidden)
        assert (part[:real] == heads * D).all() and (part[real:] == 0).all()
