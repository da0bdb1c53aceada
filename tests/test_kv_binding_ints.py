"""Numbers that do not fit the C ABI's 32 bits are refused by the binding: the
foreign-function layer would drop their upper bits and call with what is left.
No GPU is needed."""
import pytest
import torch

from error_compensated_bit_amd import binding as B

WIDE = [1 << 32, (1 << 32) + 5, 1 << 31, -(1 << 31) - 1, 1 << 40]


def small_batch(**kw):
    return B.KVBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                     torch.zeros(2, 4, dtype=torch.int32), **{**dict(rows=6, max_new=4, max_len=64), **kw})


@pytest.mark.parametrize("value", WIDE)
@pytest.mark.parametrize("field", ["rows", "max_new", "max_len"])
def test_batches(field, value):
    with pytest.raises(ValueError, match=field):
        small_batch(**{field: value}).desc(torch.device("cpu"))


@pytest.mark.parametrize("value", WIDE)
@pytest.mark.parametrize("field", ["page_size", "kv_heads", "head_dim", "bits", "group"])
def test_cache_forms(field, value):
    form = dict(num_pages=4, page_size=16, kv_heads=2, head_dim=128, bits=4, group=128)
    form[field] = value if value < 0 else form[field] + value     # a good form in the lower 32 bits
    for call in (B.echo_kv_codes_bytes, B.echo_kv_params_bytes, lambda **kw: B.alloc_kv_cache(**kw, device="cpu")):
        with pytest.raises(ValueError, match=field):
            call(**form)


def test_pages_past_64_bits():
    with pytest.raises(ValueError, match="num_pages"):
        B.alloc_kv_cache((1 << 64) + 4, 16, 2, 128, device="cpu")


@pytest.mark.parametrize("value", WIDE)
@pytest.mark.parametrize("option", ["window", "sinks"])
def test_attention_options(option, value):
    c = B.alloc_kv_cache(4, 16, 2, 128, device="cpu")
    options = {**dict(window=8, sinks=0), option: value}
    with pytest.raises(ValueError, match=option):
        B.echo_kv_workspace_bytes(c, small_batch(), 4, **options)
    with pytest.raises(ValueError, match="q_heads"):
        B.echo_kv_workspace_bytes(c, small_batch(), (1 << 32) + 4)


@pytest.mark.parametrize("option", ["window", "sinks"])
def test_attention_call(option, monkeypatch):
    c, b = B.alloc_kv_cache(4, 16, 2, 128, device="cpu"), small_batch()
    monkeypatch.setattr(B, "_kv_call", lambda cache, batch, stream: (torch.device("cpu"), cache.desc(),
                                                                     batch.desc(cache.device), 0))
    q, work = torch.zeros(6, 4, 128, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match=option):
        B.prepare_kv_attention(c, b, q, torch.zeros_like(q), 0.1, workspace=work, **{**dict(window=8), option: 1 << 32})
