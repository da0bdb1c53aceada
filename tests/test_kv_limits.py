"""Limits of the quantized K/V cache calls without a GPU: sizes just past what a
dispatch holds or 64-bit offsets reach are refused by the host."""
import pytest

from error_compensated_bit_amd import binding as B
from test_kv_abi import attention, batch, cache, qrows, ref, rows


# kv_heads * seqs * blocks of 256 rows (128 elements), 128 rows (256 elements and 64) of waves * 64 threads
@pytest.mark.parametrize("head_dim,group,row_block,threads", [(128, 128, 256, 512), (256, 128, 128, 512), (64, 64, 128, 256)])
def test_attention_grids(head_dim, group, row_block, threads):
    L, seqs, heads, per = B.load_library(), 65535, 8, 4
    most = (2 ** 32 - 1) // threads // (seqs * heads)           # blocks of rows that a dispatch holds
    new = (most + 1) * row_block // per
    form = dict(head_dim=head_dim, group=group, kv_heads=heads)
    b = batch(seqs=seqs, rows=new, max_new=new, max_len=64)
    stride = dict(row_stride=heads * per * head_dim, head_stride=head_dim)
    assert attention(L, c=cache(**form), b=b, heads=heads * per, q=qrows(**stride), out=qrows(**stride)) == B.ECHO_ERR_SHAPE
    assert L.echo_kv_workspace_bytes(cache(**form), b, heads * per, 1, 0, 0) == 0


@pytest.mark.parametrize("fault", [dict(row_stride=1 << 40), dict(row_stride=1 << 20), dict(row_stride=4096),
                                   dict(head_stride=1 << 40)])
def test_arrays_larger_than_any_memory(fault):
    """Strides whose product with the rows or heads passes 2^40 elements, and at
    the far end 64 bits of bytes."""
    L = B.load_library()
    form = dict(kv_heads=4, head_dim=128)
    b = batch(seqs=1, rows=1 << 29, max_new=64, max_len=64)
    stride = {**dict(row_stride=1024, head_stride=128), **fault}
    small = batch(seqs=1, rows=64, max_new=64, max_len=64)
    for call in (L.echo_kv_write, L.echo_kv_read):
        assert call(cache(**form), b, rows(**stride), rows(**stride), None) == B.ECHO_ERR_ARG
    assert attention(L, c=cache(**form), b=b, heads=4, q=qrows(**stride), out=qrows(row_stride=512)) == B.ECHO_ERR_ARG
    if "row_stride" in fault and fault["row_stride"] == 1 << 40:
        assert L.echo_kv_write(cache(**form), small, rows(**stride), rows(**stride), None) == B.ECHO_ERR_ARG


def test_reading_keys_and_values_into_one_array():
    """Two results in the same place would leave either: refused.  Writing both from one array is fine."""
    L = B.load_library()
    assert L.echo_kv_read(cache(), batch(), rows(), rows(), None) == B.ECHO_ERR_ARG
    assert L.echo_kv_read(cache(), batch(), rows(), rows(data=0x10000 + 8), None) == B.ECHO_ERR_ALIGN
