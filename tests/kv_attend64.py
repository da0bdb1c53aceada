"""Attention over the quantized K/V cache in 64 bits for query rows at given
positions, and caches of which only chosen positions have been written."""
from __future__ import annotations

import numpy as np
import torch

import kv_testutil as U
from error_compensated_bit_amd import binding as B


def attend_at(q, pos, k, v, causal, window, sinks, scale, spread, there=None):
    """Rows q [n, Hq, D] at positions pos [n] over the keys and values
    [length, Hk, D]; there [length]: which keys exist.  Returns the outputs and
    kv_testutil.attend's bound (see there for its derivation) with one term more.
    A probability of 1 enters the products as 2^10 at least, a step s as s / E with
    the power of two E above the largest step S, E <= 2 S.  Subnormal halves are
    off by 2^-25 at most, so each key adds 2^-35 |zero + h step| <= 2^-35 (max|v| + S h)
    and 2^-35 2 S |code - h| <= 2^-35 2 S h at most, h = 2^(bits - 1), S h = max(spread)
    (some code of the group with the largest step is 0).  Where one key has all the
    weight and its value is 0, nothing else is left."""
    n, Hq, D = q.shape
    length, Hk = k.shape[:2]
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    subnormal = 2.0 ** -35 * (np.abs(v).max(initial=0.0) + 3 * spread.max(initial=0.0))
    for i in range(n):
        see = U.visible(int(pos[i]), length, causal, window, sinks)
        if there is not None:
            see = see & there
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
            bound[i, h] = 2.0 ** -11 * (w @ sp) + (w * (err + err.max())) @ (np.abs(vv) + 2 * sp) + \
                len(s) * subnormal
    return out, bound


class Sequences:
    """Drawn keys and values for positions 0 .. lens[b] - 1 of every sequence, a
    cache filled with one byte, and pages of all of them in one table."""

    def __init__(self, lens, heads=2, per=4, D=128, bits=4, group=128, page=16, dtype="bf16", seed=0, fill=0xFF,
                 device="cuda:0", v_scale=1.0):
        self.lay = U.Layout(lens, lens, page, seed=seed, device=device)
        self.lens, self.heads, self.per, self.D, self.bits, self.group = list(lens), heads, per, D, bits, group
        self.dtype, self.device, self.scale, self.seed = dtype, device, D ** -0.5, seed
        self.cache = B.alloc_kv_cache(self.lay.pages, page, heads, D, bits, group, device)
        for t in (self.cache.k_codes, self.cache.v_codes, self.cache.k_params, self.cache.v_params):
            t.view(torch.uint8).fill_(fill)
        self.kv = [[U.draw((n, heads, D), seed + 100 * b + i, dtype, s) for i, s in ((1, 1.0), (2, v_scale))]
                   for b, n in enumerate(lens)]

    def ints(self, a):
        return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to(self.device)

    def batch(self, new, lens, rows=None, max_new=None, max_len=None, table=None):
        start = np.concatenate([[0], np.cumsum(new)])
        return B.KVBatch(self.ints(start), self.ints(lens), self.ints(self.lay.table if table is None else table),
                         rows=int(start[-1]) if rows is None else rows,
                         max_new=max(new) if max_new is None else max_new, max_len=max(lens) if max_len is None else max_len)

    def write(self, ranges):
        """Positions ranges[b] = (from, to) of every sequence into the cache."""
        new = [b - a for a, b in ranges]
        k, v = (torch.cat([self.kv[s][i][a:b] for s, (a, b) in enumerate(ranges)]).to(self.device) for i in range(2))
        B.echo_kv_write(self.cache, self.batch(new, [b for _, b in ranges]), k, v)

    def queries(self, rows, scale=1.5):
        return U.draw((rows, self.heads * self.per, self.D), self.seed + 77, self.dtype, scale)

    def check(self, got, q, b, pos, keys, causal=True, window=0, sinks=0, scale=None, there=None):
        """got, q [n, Hq, D]: rows of sequence b at positions pos, of which the first `keys` positions exist."""
        eps = torch.finfo(U.DTYPES[self.dtype]).eps
        (_, _, _), (vc, vs, _) = quantized = [U.quantize(U.host64(x[:keys]), self.bits, self.group) for x in self.kv[b]]
        k, v = (U.values(*x, self.group) for x in quantized)
        spread = np.abs(vc.astype(np.float64) - 2 ** (self.bits - 1)) * np.repeat(vs, self.group, axis=-1)
        want, bound = attend_at(U.host64(q), pos, k, v, causal, window, sinks, self.scale if scale is None else scale,
                                spread, there)
        got = U.host64(got)
        assert np.isfinite(got).all(), (b, "not finite")
        off = np.abs(got - want)
        allowed = bound + eps / 2 * (np.abs(want) + bound) + (2.0 ** -25 if self.dtype == "f16" else 2.0 ** -134)
        assert (off <= allowed).all(), (b, (off / allowed).max(), off.max())
