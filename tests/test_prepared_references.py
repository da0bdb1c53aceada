"""A prepared call keeps the memory it points at: replacing a tensor in a
payload, a cache or a batch afterwards frees nothing that the call still uses.
No call is made, and no GPU is needed."""
import gc
import weakref

import pytest
import torch

from error_compensated_bit_amd import binding as B

CPU = torch.device("cpu")


@pytest.fixture
def on_cpu(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type("S", (), {"cuda_stream": 0})())
    cpu = type("D", (), {"type": "cuda", "index": 0, "__eq__": lambda self, other: other == CPU,
                         "__ne__": lambda self, other: other != CPU, "__hash__": object.__hash__})()
    monkeypatch.setattr(B.KVCache, "device", property(lambda self: cpu))
    monkeypatch.setattr(torch.Tensor, "device", property(lambda self: cpu))


def held(owner, name):
    """A weak reference to the tensor's memory, and the tensor replaced in its owner."""
    t = getattr(owner, name)
    ref = weakref.ref(t)
    setattr(owner, name, None)
    return ref


def test_cache_and_batch(on_cpu):
    for kind in ("write", "read", "attention"):
        c = B.alloc_kv_cache(4, 16, 2, 128, device="cpu")
        b = B.KVBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                      torch.zeros(2, 4, dtype=torch.int32), rows=6, max_new=4, max_len=64)
        k, v, q, out = (torch.zeros(6, h, 128, dtype=torch.bfloat16) for h in (2, 2, 4, 4))
        work = torch.zeros(64, dtype=torch.uint8)
        if kind == "attention":
            call = B.prepare_kv_attention(c, b, q, out, 0.1, workspace=work, stream=0)
        else:
            call = getattr(B, f"prepare_kv_{kind}")(c, b, k, v, stream=0)
        refs = [held(c, n) for n in ("k_codes", "v_codes", "k_params", "v_params")]
        refs += [held(b, n) for n in ("row_start", "kv_len", "page_table")]
        gc.collect()
        assert all(r() is not None for r in refs), kind
        del call
        gc.collect()
        assert all(r() is None for r in refs), kind


def test_payloads():
    cfg = B.make_config()
    x, state = torch.zeros(1024, dtype=torch.bfloat16), torch.zeros(2048)
    for kind in ("entry", "owner", "gather"):
        pays = [B.alloc_payload(512, 4, "cpu") for _ in range(3)]
        if kind == "entry":
            call = B.prepare_quantize_feedback(cfg, 2, 0, 1024, x, state, pays[:2], stream=0)
        elif kind == "owner":
            call = B.prepare_owner_reduce_requant(cfg, 2, 0, 1024, x, state, pays[:2], pays[2], stream=0)
        else:
            call = B.prepare_dequant_gather(cfg, 2, 1024, pays[:2], x, stream=0)
        used = pays if kind == "owner" else pays[:2]
        refs = [held(p, n) for p in used for n in ("codes", "params")]
        gc.collect()
        assert all(r() is not None for r in refs), kind
        del call
        gc.collect()
        assert all(r() is None for r in refs), kind
