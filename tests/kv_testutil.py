"""Helpers of the quantized K/V cache tests: plain caches, batches and the
operators' definitions in 64 bits.  Nothing here imports the kernels' code."""
from __future__ import annotations

import math

import numpy as np
import torch

from error_compensated_bit_amd import binding as B

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def f16(x):
    with np.errstate(over="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float16).astype(np.float64)


def quantize(x: np.ndarray, bits: int, group: int):
    """Codes, steps and zeros of rows [..., D] by the definition: 64-bit
    arithmetic, rounded to binary32 or binary16 after every operation.
    fmin/fmax ignore NaN; a group of NaN only has the lowest zero."""
    top = float(2 ** bits - 1)
    v = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // group, group)
    with np.errstate(all="ignore"):
        low = np.fmin.reduce(v, axis=-1, keepdims=True)
        high = np.fmax.reduce(v, axis=-1, keepdims=True)
        zero = f16(np.fmin(np.fmax(low, -65504.0), 65504.0)) + 0.0
        step = f32(f32(high - zero) / top)
        step = f16(np.where(step > 0, np.fmin(step, 65504.0), 0.0))
        inv = f32(np.where(step > 0, 1.0 / step, 0.0))
        code = np.fmin(np.fmax(np.rint(f32(f32(v - zero) * inv)), 0.0), top)
    return code.reshape(x.shape).astype(np.uint8), step[..., 0], zero[..., 0]


def values(code, step, zero, group):
    c = code.astype(np.float64).reshape(*code.shape[:-1], code.shape[-1] // group, group)
    return f32(c * step[..., None] + zero[..., None]).reshape(code.shape)


def key_order(D):
    """Element stored at each place of a key row."""
    e = np.empty(D, np.int64)
    for w in range(D // 32):
        for quad in range(4):
            place = (quad * (D // 32) + w) * 8
            e[place:place + 8] = 32 * w + 8 * quad + np.arange(8)
    return e


def value_order(D):
    e = np.empty(D, np.int64)
    for m in range(16):
        for i in range(D // 16):
            e[m * (D // 16) + i] = 16 * i + m
    return e


def unpack(codes: np.ndarray, bits: int, order: np.ndarray) -> np.ndarray:
    """Codes by element from stored rows [..., bytes]."""
    if bits == 4:
        stored = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    else:
        stored = codes
    out = np.empty_like(stored)
    out[..., order] = stored
    return out


def unpack_params(words: np.ndarray):
    w = words.view(np.uint32)
    return ((w & 0xFFFF).astype(np.uint16).view(np.float16).astype(np.float64),
            (w >> 16).astype(np.uint16).view(np.float16).astype(np.float64))


def cache_rows(cache: B.KVCache):
    """(codes, step, zero) of keys and values by element: [pages, heads, slots, D]."""
    out = []
    for codes, params, order in ((cache.k_codes, cache.k_params, key_order(cache.head_dim)),
                                 (cache.v_codes, cache.v_params, value_order(cache.head_dim))):
        step, zero = unpack_params(params.cpu().numpy())
        out.append((unpack(codes.cpu().numpy(), cache.bits, order), step, zero))
    return out


class Layout:
    """Sequences with `new` rows each and `lens` positions, pages scattered over a cache."""

    def __init__(self, lens, new, page, spare=2, seed=0, entries=None, device="cuda:0"):
        self.lens, self.new, self.page = list(lens), list(new), page
        need = [-(-n // page) for n in self.lens]
        self.pages = sum(need) + spare
        order = np.random.default_rng(seed).permutation(self.pages)
        width = entries or max(need + [1])
        self.table = np.full((len(self.lens), width), -1, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.rows = int(self.start[-1])
        self.device = device

    def batch(self, new=None, rows=None, max_new=None, max_len=None) -> B.KVBatch:
        new = self.new if new is None else list(new)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        t = [torch.from_numpy(np.ascontiguousarray(a)).to(self.device)
             for a in (start, np.asarray(self.lens, np.int32), self.table)]
        return B.KVBatch(*t, rows=int(start[-1]) if rows is None else rows,
                         max_new=max(list(new) + [0]) if max_new is None else max_new,
                         max_len=max(self.lens + [0]) if max_len is None else max_len)

    def slots(self, b, positions):
        positions = np.asarray(positions)
        return self.table[b, positions // self.page], positions % self.page


def draw(shape, seed, dtype="bf16", scale=1.0, offset=0.0):
    """Host values of a 16- or 32-bit type, as a torch tensor."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + offset).to(DTYPES[dtype])


def host64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def visible(pos, length, causal, window, sinks):
    j = np.arange(length)
    if not causal:
        return np.ones(length, bool)
    see = j <= pos
    if window:
        see &= (pos - j < window) | (j < sinks)
    return see


def attend(q, k, v, length, causal, window, sinks, scale, spread):
    """64-bit attention of the n last positions' queries q [n, Hq, D] over keys
    and values [length, Hk, D], and the bound of the error that the kernel's
    number formats allow, without the output's own rounding.

    spread [length, Hk, D]: step * |code - half|, what a probability is
    multiplied with when it has been rounded to f16 (half a step: 2^-11
    relative, or 2^-25 of the largest product once it is subnormal, which is
    2^-35 of p = 1 and left to the last term).  The last term covers binary32:
    a score's relative error is at most (D + 8) 2^-23 of the sum of its terms'
    magnitudes, and enters a probability by its absolute size; the exponential
    and sums of n terms add (n / 32 + 16) 2^-23 of the sum of magnitudes."""
    n, Hq, D = q.shape
    Hk = k.shape[1]
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        see = visible(length - n + i, length, causal, window, sinks)
        if not see.any():
            continue
        for h in range(Hq):
            kk, vv, sp = (a[see, h * Hk // Hq] for a in (k, v, spread))
            s = scale * (kk @ q[i, h])
            size = abs(scale) * (np.abs(kk) @ np.abs(q[i, h]))
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ vv
            err = size * (D + 8) * 2.0 ** -23 + (len(s) / 32 + 16) * 2.0 ** -23
            mag = np.abs(vv) + 2 * sp
            bound[i, h] = 2.0 ** -11 * (w @ sp) + (w * (err + err.max())) @ mag
    return out, bound
