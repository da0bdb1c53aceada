"""ctypes binding of libecho_amd.so (include/echo.h), same names as the C ABI.

Argument marshalling only: torch tensors are passed as device pointers and
host descriptor arrays are built for the payload tables.  Every step of the
all-reduce share runs in the library's kernels; there is no fallback: if the
library is not built, loading it raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

from .build import library_path

# constants of include/echo.h
ECHO_OK, ECHO_ERR_ARG, ECHO_ERR_SHAPE, ECHO_ERR_ALIGN, ECHO_ERR_HIP = 0, -1, -2, -3, -4
ECHO_IN_BF16, ECHO_IN_F16 = 0, 1
ECHO_OUT_BF16, ECHO_OUT_F32 = 0, 1
ECHO_STATE_F32, ECHO_STATE_BF16 = 0, 1
ECHO_MAX_RANKS = 16
ECHO_GROUP = 128
ECHO_KV_BF16, ECHO_KV_F16, ECHO_KV_F32 = 0, 1, 2

EXPORTED = ("echo_state_reset", "echo_quantize_feedback", "echo_owner_reduce_requant",
            "echo_dequant_gather", "echo_segment_len", "echo_codes_bytes", "echo_params_bytes",
            "echo_state_bytes", "echo_error_string",
            "echo_kv_write", "echo_kv_read", "echo_kv_attention",
            "echo_kv_codes_bytes", "echo_kv_params_bytes", "echo_kv_workspace_bytes")


class echo_config(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32), ("eta", ctypes.c_float),
                ("beta_short", ctypes.c_float), ("beta_long", ctypes.c_float),
                ("mix_long", ctypes.c_float)]


class echo_seg(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("params", ctypes.c_void_p)]


class echo_kv_cache(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_params", ctypes.c_void_p), ("v_params", ctypes.c_void_p)]


class echo_kv_batch(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int32), ("rows", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("max_len", ctypes.c_int32), ("table_stride", ctypes.c_int64),
                ("row_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p)]


class echo_kv_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class EchoError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {error_string(code)} (code {code})")
        self.code = code


_LIB = None


def load_library() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build the HIP library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(path)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        cfgp, segp = ctypes.POINTER(echo_config), ctypes.POINTER(echo_seg)
        L.echo_state_reset.argtypes = [cfgp, vp, i64, vp]
        L.echo_quantize_feedback.argtypes = [cfgp, i32, i32, i64, vp, vp, segp, vp]
        L.echo_owner_reduce_requant.argtypes = [cfgp, i32, i32, i64, vp, vp, segp, segp, vp]
        L.echo_dequant_gather.argtypes = [cfgp, i32, i64, segp, vp, vp]
        L.echo_codes_bytes.argtypes = [i64, i32]
        L.echo_params_bytes.argtypes = [i64, i32]
        L.echo_state_bytes.argtypes = [i64, i32]
        L.echo_segment_len.argtypes = [i64, i32, i32]
        L.echo_segment_len.restype = ctypes.c_int64
        L.echo_codes_bytes.restype = ctypes.c_size_t
        L.echo_params_bytes.restype = ctypes.c_size_t
        L.echo_state_bytes.restype = ctypes.c_size_t
        L.echo_error_string.argtypes = [i32]
        L.echo_error_string.restype = ctypes.c_char_p
        cachep, batchp, rowsp = (ctypes.POINTER(t) for t in (echo_kv_cache, echo_kv_batch, echo_kv_rows))
        L.echo_kv_write.argtypes = [cachep, batchp, rowsp, rowsp, vp]
        L.echo_kv_read.argtypes = [cachep, batchp, rowsp, rowsp, vp]
        L.echo_kv_attention.argtypes = [cachep, batchp, i32, rowsp, rowsp, ctypes.c_float, i32, i32, i32,
                                        vp, ctypes.c_size_t, vp]
        L.echo_kv_codes_bytes.argtypes = [cachep]
        L.echo_kv_params_bytes.argtypes = [cachep]
        L.echo_kv_workspace_bytes.argtypes = [cachep, batchp, i32, i32, i32, i32]
        for name in ("echo_kv_codes_bytes", "echo_kv_params_bytes", "echo_kv_workspace_bytes"):
            getattr(L, name).restype = ctypes.c_size_t
        for name in ("echo_state_reset", "echo_quantize_feedback",
                     "echo_owner_reduce_requant", "echo_dequant_gather",
                     "echo_kv_write", "echo_kv_read", "echo_kv_attention"):
            getattr(L, name).restype = ctypes.c_int
        _LIB = L
    return _LIB


def error_string(code: int) -> str:
    return load_library().echo_error_string(code).decode()


def make_config(bits=4, group=ECHO_GROUP, eta=1.0, beta_short=0.5, beta_long=0.9,
                mix_long=1.0 / 80.0, in_dtype=ECHO_IN_BF16, out_dtype=ECHO_OUT_BF16,
                state_dtype=ECHO_STATE_F32) -> echo_config:
    return echo_config(bits, group, in_dtype, out_dtype, state_dtype, eta, beta_short,
                       beta_long, mix_long)


@dataclass
class Payload:
    """One segment's payload: codes (uint8) and params (int32 words, scale | zero << 16)."""
    codes: torch.Tensor
    params: torch.Tensor

    def tensors(self) -> tuple:
        return self.codes, self.params

    def seg(self) -> echo_seg:
        return echo_seg(_ptr(self.codes), _ptr(self.params))


def echo_codes_bytes(seg_len: int, bits: int) -> int:
    return load_library().echo_codes_bytes(seg_len, bits)


def echo_params_bytes(seg_len: int, group: int = ECHO_GROUP) -> int:
    return load_library().echo_params_bytes(seg_len, group)


def echo_segment_len(n: int, P: int, group: int = ECHO_GROUP) -> int:
    return load_library().echo_segment_len(n, P, group)


def echo_state_bytes(n: int, state_dtype: int) -> int:
    return load_library().echo_state_bytes(n, state_dtype)


def alloc_payload(seg_len: int, bits: int, device, fill: int | None = None,
                  group: int = ECHO_GROUP) -> Payload:
    """Payload buffers for seg_len elements; `fill` sets every byte (sentinels)."""
    cb, pb = echo_codes_bytes(seg_len, bits), echo_params_bytes(seg_len, group)
    if cb == 0 or pb == 0:
        raise ValueError(f"no payload layout for {seg_len} elements at {bits} bits")
    if fill is None:
        return Payload(torch.empty(cb, dtype=torch.uint8, device=device),
                       torch.empty(pb // 4, dtype=torch.int32, device=device))
    return Payload(torch.full((cb,), fill, dtype=torch.uint8, device=device),
                   torch.full((pb,), fill, dtype=torch.uint8, device=device).view(torch.int32))


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("echo buffers must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _seg_table(P: int, payloads) -> ctypes.Array:
    tab = (echo_seg * P)()
    for p, pay in enumerate(payloads):
        if pay is not None:
            tab[p] = pay.seg()
    return tab


def _check(rc: int, where: str):
    if rc != ECHO_OK:
        raise EchoError(rc, where)


def echo_state_reset(cfg: echo_config, state: torch.Tensor, n: int, stream=None):
    """state: 2n elements (S_j, L_j pairs) of the config's state type."""
    _check(load_library().echo_state_reset(ctypes.byref(cfg), _ptr(state), n, _stream(stream)),
           "echo_state_reset")


def echo_quantize_feedback(cfg: echo_config, P: int, rank: int, n: int, x: torch.Tensor,
                           state: torch.Tensor, out, stream=None):
    """out: list of P Payloads (entry `rank` may be None)."""
    _check(load_library().echo_quantize_feedback(ctypes.byref(cfg), P, rank, n, _ptr(x),
                                                 _ptr(state), _seg_table(P, out), _stream(stream)),
           "echo_quantize_feedback")


def echo_owner_reduce_requant(cfg: echo_config, P: int, rank: int, n: int, x: torch.Tensor,
                              state: torch.Tensor, inp, out: Payload, stream=None):
    """inp: list of P Payloads received for segment `rank` (entry `rank` may be None)."""
    out_seg = out.seg()
    _check(load_library().echo_owner_reduce_requant(ctypes.byref(cfg), P, rank, n, _ptr(x),
                                                    _ptr(state), _seg_table(P, inp),
                                                    ctypes.byref(out_seg), _stream(stream)),
           "echo_owner_reduce_requant")


def echo_dequant_gather(cfg: echo_config, P: int, n: int, inp, out: torch.Tensor, stream=None):
    """inp: list of the P owners' requantized Payloads, in segment order."""
    _check(load_library().echo_dequant_gather(ctypes.byref(cfg), P, n, _seg_table(P, inp),
                                              _ptr(out), _stream(stream)),
           "echo_dequant_gather")


class Prepared:
    """One entry-point call with every argument marshalled once (config,
    payload tables, pointers and stream): calling it makes only the foreign
    call.  For callers that repeat the same call on the same buffers, where
    marshalling would cost more host time than a small message's kernels.
    It holds references to every tensor it was given (the tensors themselves:
    a payload, cache or batch may be given others afterwards), so they stay
    allocated while it exists; it always launches on the stream it was prepared
    with."""

    def __init__(self, fn, args, keep, where: str):
        self._fn = fn
        self._args = args
        self._keep = keep          # the ctypes objects the byref arguments point at
        self._where = where

    def __call__(self):
        rc = self._fn(*self._args)
        if rc != ECHO_OK:
            raise EchoError(rc, self._where)


def prepare_quantize_feedback(cfg: echo_config, P: int, rank: int, n: int, x: torch.Tensor,
                              state: torch.Tensor, out, stream=None) -> Prepared:
    L = load_library()
    c = echo_config(*(getattr(cfg, f) for f, _ in echo_config._fields_))
    return Prepared(L.echo_quantize_feedback,
                    (ctypes.byref(c), P, rank, n, _ptr(x), _ptr(state), _seg_table(P, out),
                     _stream(stream)), (c, x, state, [p.tensors() for p in out if p]), "echo_quantize_feedback")


def prepare_owner_reduce_requant(cfg: echo_config, P: int, rank: int, n: int, x: torch.Tensor,
                                 state: torch.Tensor, inp, out: Payload, stream=None) -> Prepared:
    L = load_library()
    c = echo_config(*(getattr(cfg, f) for f, _ in echo_config._fields_))
    out_seg = out.seg()
    return Prepared(L.echo_owner_reduce_requant,
                    (ctypes.byref(c), P, rank, n, _ptr(x), _ptr(state), _seg_table(P, inp),
                     ctypes.byref(out_seg), _stream(stream)), (c, out_seg, x, state, [p.tensors() for p in (*inp, out) if p]),
                    "echo_owner_reduce_requant")


def prepare_dequant_gather(cfg: echo_config, P: int, n: int, inp, out: torch.Tensor,
                           stream=None) -> Prepared:
    L = load_library()
    c = echo_config(*(getattr(cfg, f) for f, _ in echo_config._fields_))
    return Prepared(L.echo_dequant_gather,
                    (ctypes.byref(c), P, n, _seg_table(P, inp), _ptr(out), _stream(stream)),
                    (c, [p.tensors() for p in inp if p], out), "echo_dequant_gather")


# ------------------------------------------------------------------ quantized K/V cache
_INT32 = 1 << 31


def _int(width: int, /, **values):
    """Refuse what a signed integer of that width does not hold: ctypes would
    pass its lower bits.  (The calls of a step compare with _INT32 first.)"""
    for name, v in values.items():
        if not -(1 << width - 1) <= v < 1 << width - 1:
            raise ValueError(f"{name}: {v} does not fit {width} bits")


_KV_DTYPES = {torch.bfloat16: ECHO_KV_BF16, torch.float16: ECHO_KV_F16, torch.float32: ECHO_KV_F32}


@dataclass
class KVCache:
    """A paged cache of quantized keys and values (see include/echo.h for the
    order of the codes inside a row).  codes: uint8 [num_pages, kv_heads,
    page_size, head_dim * bits / 8]; params: int32 words [num_pages, kv_heads,
    page_size, head_dim / group], scale | zero << 16."""
    bits: int
    group: int
    head_dim: int
    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_params: torch.Tensor
    v_params: torch.Tensor

    @property
    def num_pages(self) -> int:
        return self.k_codes.shape[0]

    @property
    def kv_heads(self) -> int:
        return self.k_codes.shape[1]

    @property
    def page_size(self) -> int:
        return self.k_codes.shape[2]

    @property
    def device(self) -> torch.device:
        return self.k_codes.device

    def tensors(self) -> tuple:
        return self.k_codes, self.v_codes, self.k_params, self.v_params

    def desc(self) -> echo_kv_cache:
        pages, heads, slots = self.k_codes.shape[:3]
        want = {"codes": ((pages, heads, slots, self.head_dim * self.bits // 8), torch.uint8),
                "params": ((pages, heads, slots, self.head_dim // self.group), torch.int32)}
        for name in ("k_codes", "v_codes", "k_params", "v_params"):
            t = getattr(self, name)
            shape, dtype = want[name[2:]]
            if tuple(t.shape) != shape or t.dtype != dtype or t.device != self.device:
                raise ValueError(f"{name}: expected {dtype} {shape} on {self.device}, "
                                 f"got {t.dtype} {tuple(t.shape)} on {t.device}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if max(self.bits, self.group, self.head_dim) >= _INT32 or min(self.bits, self.group, self.head_dim) < -_INT32:
            _int(32, bits=self.bits, group=self.group, head_dim=self.head_dim)
        return echo_kv_cache(self.bits, self.group, self.head_dim, heads, slots, 0, pages, _ptr(self.k_codes),
                             _ptr(self.v_codes), _ptr(self.k_params), _ptr(self.v_params))


@dataclass
class KVBatch:
    """The rows of one call: sequence b has rows row_start[b] .. row_start[b + 1] - 1
    of the packed arrays, its last positions of kv_len[b]; page_table [seqs,
    entries] names their pages.  All int32 on the GPU.  rows: rows of the packed
    arrays; max_new, max_len: upper bounds of a sequence's rows and length."""
    row_start: torch.Tensor
    kv_len: torch.Tensor
    page_table: torch.Tensor
    rows: int
    max_new: int
    max_len: int

    def tensors(self) -> tuple:
        return self.row_start, self.kv_len, self.page_table

    def desc(self, device: torch.device) -> echo_kv_batch:
        seqs = self.kv_len.numel()
        if self.page_table.dim() != 2 or self.page_table.shape[0] != seqs or self.row_start.shape != (seqs + 1,) \
                or self.kv_len.dim() != 1:
            raise ValueError("a batch is row_start [seqs + 1], kv_len [seqs] and page_table [seqs, entries]")
        for t in (self.row_start, self.kv_len, self.page_table):
            if t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
                raise ValueError(f"a batch's arrays are contiguous int32 on the cache's device {device}")
        if max(self.rows, self.max_new, self.max_len) >= _INT32 or min(self.rows, self.max_new, self.max_len) < -_INT32:
            _int(32, rows=self.rows, max_new=self.max_new, max_len=self.max_len)
        return echo_kv_batch(seqs, self.rows, self.max_new, self.max_len, self.page_table.shape[1],
                             _ptr(self.row_start), _ptr(self.kv_len), _ptr(self.page_table))


def _kv_form(num_pages, page_size, kv_heads, head_dim, bits, group) -> echo_kv_cache:
    _int(32, bits=bits, group=group, head_dim=head_dim, kv_heads=kv_heads, page_size=page_size)
    _int(64, num_pages=num_pages)
    return echo_kv_cache(bits, group, head_dim, kv_heads, page_size, 0, num_pages, None, None, None, None)


def echo_kv_codes_bytes(num_pages: int, page_size: int, kv_heads: int, head_dim: int, bits: int = 4,
                        group: int = ECHO_GROUP) -> int:
    return load_library().echo_kv_codes_bytes(ctypes.byref(
        _kv_form(num_pages, page_size, kv_heads, head_dim, bits, group)))


def echo_kv_params_bytes(num_pages: int, page_size: int, kv_heads: int, head_dim: int, bits: int = 4,
                         group: int = ECHO_GROUP) -> int:
    return load_library().echo_kv_params_bytes(ctypes.byref(
        _kv_form(num_pages, page_size, kv_heads, head_dim, bits, group)))


def alloc_kv_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, bits: int = 4,
                   group: int = ECHO_GROUP, device="cuda") -> KVCache:
    if echo_kv_codes_bytes(num_pages, page_size, kv_heads, head_dim, bits, group) == 0:
        raise ValueError(f"no cache of {num_pages} pages of {page_size} slots, {kv_heads} heads of {head_dim} "
                         f"elements at {bits} bits in groups of {group}")
    lead = (num_pages, kv_heads, page_size)
    codes = [torch.empty(*lead, head_dim * bits // 8, dtype=torch.uint8, device=device) for _ in "kv"]
    params = [torch.empty(*lead, head_dim // group, dtype=torch.int32, device=device) for _ in "kv"]
    return KVCache(bits, group, head_dim, *codes, *params)


def _kv_rows(t: torch.Tensor, what: str, rows: int, heads: int, head_dim: int, device: torch.device) -> echo_kv_rows:
    if tuple(t.shape) != (rows, heads, head_dim) or t.device != device or t.dtype not in _KV_DTYPES:
        raise ValueError(f"{what}: expected bf16, fp16 or fp32 rows ({rows}, {heads}, {head_dim}) on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.numel() and t.stride(2) != 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    return echo_kv_rows(t.data_ptr() or None, t.stride(0), t.stride(1), _KV_DTYPES[t.dtype], 0)


class _PreparedOn(Prepared):
    """A prepared call of tensors on one device: made with that device current,
    whichever device the caller has current."""

    def __init__(self, fn, args, keep, where: str, device: torch.device):
        super().__init__(fn, args, keep, where)
        self._device = device.index

    def __call__(self):
        if torch.cuda.current_device() == self._device:
            return super().__call__()
        with torch.cuda.device(self._device):
            return super().__call__()


def _kv_call(cache: KVCache, batch: KVBatch, stream):
    device = cache.device
    if device.type != "cuda":
        raise ValueError("the cache must be on a GPU")
    st = torch.cuda.current_stream(device).cuda_stream if stream is None else _stream(stream)
    return device, cache.desc(), batch.desc(device), st


def _prepare_kv_rows(fn, where: str, cache: KVCache, batch: KVBatch, k, v, stream) -> Prepared:
    device, c, b, st = _kv_call(cache, batch, stream)
    kr, vr = (_kv_rows(t, n, batch.rows, cache.kv_heads, cache.head_dim, device) for t, n in ((k, "k"), (v, "v")))
    return _PreparedOn(fn, (ctypes.byref(c), ctypes.byref(b), ctypes.byref(kr), ctypes.byref(vr), st),
                       (c, b, kr, vr, cache.tensors(), batch.tensors(), k, v), where, device)


def prepare_kv_write(cache: KVCache, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, stream=None) -> Prepared:
    return _prepare_kv_rows(load_library().echo_kv_write, "echo_kv_write", cache, batch, k, v, stream)


def prepare_kv_read(cache: KVCache, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, stream=None) -> Prepared:
    return _prepare_kv_rows(load_library().echo_kv_read, "echo_kv_read", cache, batch, k, v, stream)


def echo_kv_workspace_bytes(cache: KVCache, batch: KVBatch, q_heads: int, causal=True, window: int = 0,
                            sinks: int = 0) -> int:
    c, b = cache.desc(), batch.desc(cache.device)
    _int(32, q_heads=q_heads, window=window, sinks=sinks)
    return load_library().echo_kv_workspace_bytes(ctypes.byref(c), ctypes.byref(b), q_heads, int(causal), window,
                                                  sinks)


def prepare_kv_attention(cache: KVCache, batch: KVBatch, q: torch.Tensor, out: torch.Tensor, scale: float,
                         causal=True, window: int = 0, sinks: int = 0, workspace: torch.Tensor | None = None,
                         stream=None) -> Prepared:
    """workspace: uint8, at least echo_kv_workspace_bytes(), zeros; by default one
    of the prepared call's own.  Calls that may run at the same time (other
    streams, graphs replayed side by side) must not share one."""
    device, c, b, st = _kv_call(cache, batch, stream)
    if max(window, sinks) >= _INT32 or min(window, sinks) < -_INT32:
        _int(32, window=window, sinks=sinks)
    q_heads = q.shape[1] if q.dim() == 3 else 0
    qr, outr = (_kv_rows(t, n, batch.rows, q_heads, cache.head_dim, device) for t, n in ((q, "q"), (out, "out")))
    if workspace is None:
        with torch.cuda.stream(_as_stream(device, stream)):
            room = load_library().echo_kv_workspace_bytes(ctypes.byref(c), ctypes.byref(b), q_heads, int(causal), window,
                                                          sinks)
            workspace = torch.zeros(room, dtype=torch.uint8, device=device)
    elif workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: contiguous uint8 on {device}")
    return _PreparedOn(load_library().echo_kv_attention,
                       (ctypes.byref(c), ctypes.byref(b), q_heads, ctypes.byref(qr), ctypes.byref(outr), scale,
                        int(causal), window, sinks, _ptr(workspace) or None, workspace.numel(), st),
                       (c, b, qr, outr, cache.tensors(), batch.tensors(), q, out, workspace), "echo_kv_attention", device)


def echo_kv_write(cache: KVCache, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, stream=None):
    """k, v: [rows, kv_heads, head_dim], bf16, fp16 or fp32, any strides of 16-byte multiples."""
    prepare_kv_write(cache, batch, k, v, stream)()


def echo_kv_read(cache: KVCache, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, stream=None):
    """k, v: [rows, kv_heads, head_dim] to fill, bf16, fp16 or fp32."""
    prepare_kv_read(cache, batch, k, v, stream)()


def echo_kv_attention(cache: KVCache, batch: KVBatch, q: torch.Tensor, out: torch.Tensor, scale: float,
                      causal=True, window: int = 0, sinks: int = 0, workspace: torch.Tensor | None = None,
                      stream=None):
    """q, out: [rows, q_heads, head_dim], both bf16 or both fp16.  Without a
    workspace one is allocated for this call on its stream."""
    prepare_kv_attention(cache, batch, q, out, scale, causal, window, sinks, workspace, stream)()


def _as_stream(device: torch.device, stream):
    """torch's object for a stream argument: memory allocated under it may be
    reused once the stream's work is done."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if hasattr(stream, "cuda_stream"):
        return stream
    return torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
