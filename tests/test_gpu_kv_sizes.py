"""The ends of what the quantized K/V cache calls take: more heads than a block
has rows, and packed rows past 2^32 elements."""
import numpy as np
import pytest
import torch

import kv_testutil as U
from error_compensated_bit_amd import binding as B
from kv_attend64 import Sequences, attend_at

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("heads,per,D,group", [(300, 2, 64, 64), (4096, 1, 64, 32), (1, 300, 128, 128), (3, 130, 64, 64)])
def test_many_heads(heads, per, D, group):
    s = Sequences([19, 5], heads=heads, per=per, D=D, group=group, seed=heads)
    s.write([(0, 19), (0, 5)])
    back = [torch.zeros(24, heads, D, dtype=torch.float32, device=DEV) for _ in "kv"]
    B.echo_kv_read(s.cache, s.batch([19, 5], [19, 5]), *back)
    for i in range(2):
        x = U.host64(torch.cat([s.kv[0][i], s.kv[1][i]]))
        assert np.array_equal(U.host64(back[i]), U.values(*U.quantize(x, 4, group), group))
    q = s.queries(3)
    out = torch.empty_like(q, device=DEV)
    B.echo_kv_attention(s.cache, s.batch([2, 1], [19, 5]), q.to(DEV), out, s.scale)
    s.check(out[:2], q[:2], 0, [17, 18], 19)
    s.check(out[2:], q[2:], 1, [4], 5)


def test_rows_past_32_bits():
    """One long prompt: queries, keys and values as views of one projection of 2^32 elements and more."""
    heads, D, window, rows = 8, 128, 64, (1 << 20) + 100
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough free device memory")
    x = torch.empty(rows, 32, D, dtype=torch.bfloat16, device=DEV).normal_()
    out = torch.zeros_like(x)
    table = torch.arange(-(-rows // 256), dtype=torch.int32, device=DEV).flip(0)[None].contiguous()
    cache = B.alloc_kv_cache(table.shape[1], 256, heads, D, device=DEV)
    batch = B.KVBatch(torch.tensor([0, rows], dtype=torch.int32, device=DEV),
                      torch.tensor([rows], dtype=torch.int32, device=DEV), table, rows=rows, max_new=rows, max_len=rows)
    B.echo_kv_write(cache, batch, x[:, :8], x[:, 8:16])
    B.echo_kv_read(cache, batch, out[:, 24:], out[:, 16:24])
    kv = [U.quantize(U.host64(x[-200:, i:i + 8]), 4, 128) for i in (0, 8)]
    for got, q in ((out[-200:, 24:], kv[0]), (out[-200:, 16:24], kv[1])):
        want = torch.from_numpy(U.values(*q, 128)).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)
    B.echo_kv_attention(cache, batch, x, out, D ** -0.5, window=window)
    k, v = (U.values(*q, 128) for q in kv)
    spread = np.abs(kv[1][0].astype(np.float64) - 8) * np.repeat(kv[1][1], 128, axis=-1)
    want, bound = attend_at(U.host64(x[-5:]), np.arange(195, 200), k, v, True, window, 0, D ** -0.5, spread)
    off = np.abs(U.host64(out[-5:]) - want)
    assert (off <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()
    assert out[:: 1 << 17].isfinite().all() and out[:: 1 << 17].any(-1).all()
