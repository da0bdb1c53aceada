"""The quantized K/V cache operators on realistic cases: writing rows into a
paged cache of 4- or 8-bit codes, reading rows back, and attention over it.

`run` computes them in plain torch operations (`own` false) or through the
library's entry points (`own` true); `exact` computes them in 64 bits.

Cache: every row (one token of one K/V head, `head_dim` elements) is quantized
in groups of `group` elements: zero = fp16(min), step = fp16((max - zero) /
qmax), code = round-half-even((x - zero) * (1 / step)) clamped to 0..qmax,
every operation rounded to binary32; the value of a code is code * step +
zero.  Position p of sequence b lies in slot p % page of the page
page_table[b, p // page].

Rows: sequence b brings new_b rows; they are its last positions, so row i sits
at position context_b + i of context_b + new_b.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _case(name, kind, seqs, context, context_spread, new, new_spread, q_heads, kv_heads, head_dim,
          bits=4, group=128, page=64, dtype="bf16", window=0, sinks=0, causal=True):
    return {"name": name, "kind": kind, "seqs": seqs, "context": context, "context_spread": context_spread,
            "new": new, "new_spread": new_spread, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "bits": bits, "group": min(group, head_dim), "page": page, "dtype": dtype,
            "window": window, "sinks": sinks, "causal": causal}


def listed():
    return [
        # one new token for each of 32 running sequences, put into the cache and read back: latency counts
        _case("cache_tokens", "round", 32, 1999, 1500, 1, 0, 32, 8, 128),
        # a long prompt's keys and values put into the cache and read back for a 16-bit consumer
        _case("cache_prompt", "round", 1, 0, 0, 16384, 0, 32, 8, 128),
        # ragged prompts of odd lengths, 8-bit codes in small groups, half precision, small pages
        _case("cache_ragged_8bit", "round", 13, 777, 700, 1531, 1400, 16, 16, 64, bits=8, group=32, page=16,
              dtype="f16"),
        # a long sequence's whole cache read back (moved to another worker, or given to a 16-bit kernel)
        _case("read_long", "read", 1, 0, 0, 131072, 0, 32, 8, 128),
        # one user's next token on a short context: the smallest call
        _case("token_short", "attend", 1, 512, 0, 1, 0, 32, 8, 128),
        # a server's decode step: 64 sequences of different lengths
        _case("token_batch", "attend", 64, 4095, 3000, 1, 0, 32, 8, 128),
        # next tokens on very long documents
        _case("token_long", "attend", 4, 131071, 9999, 1, 0, 32, 8, 128),
        # window and first tokens, one head for each K/V head, half precision, groups smaller than a row
        _case("token_window", "attend", 32, 32767, 20000, 1, 0, 16, 16, 128, group=32, window=4096, sinks=4,
              dtype="f16", page=32),
        # five drafted tokens verified at once on an 8-bit cache
        _case("draft_8bit", "attend", 16, 6143, 5000, 5, 0, 64, 8, 128, bits=8, group=64),
        # a chunk of a long prompt against the part of it that is in the cache already
        _case("chunk", "attend", 1, 16384, 0, 2048, 0, 32, 8, 128),
        # ragged prompts of odd lengths, half precision, small heads
        _case("prompts_ragged", "attend", 7, 0, 0, 2777, 2700, 24, 8, 64, group=64, dtype="f16", page=16),
        # a prompt under a sliding window with first tokens kept, wide heads
        _case("prompt_window", "attend", 1, 0, 0, 8192, 0, 8, 4, 256, window=1024, sinks=4),
    ]


def draw(rng):
    """One more case; never more work than the largest listed one of its kind."""
    most = {}
    for c in listed():
        w = work(c)
        for k in ("bytes", "flops"):
            most[c["kind"], k] = max(most.get((c["kind"], k), 0), w[k])

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        kind = rng.choice(["round", "round", "read", "attend", "attend", "attend"])
        D = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 5, 8, 16])
        shape = rng.choice(["tokens", "draft", "prompt"])
        new = 1 if shape == "tokens" else rng.randint(2, 9) if shape == "draft" else log(16, 16384)
        context = log(1, 131072) if shape != "prompt" or rng.random() < 0.5 else 0
        if kind == "read":
            context = 0
            new = log(1, 131072)
        seqs = log(1, 64)
        window = log(16, 8192) if kind == "attend" and rng.random() < 0.3 else 0
        c = _case("", kind, seqs, context, rng.randint(0, context) if seqs > 1 else 0, new,
                  rng.randint(0, new - 1) if seqs > 1 else 0, kv_heads * rng.choice([1, 2, 3, 4, 8]), kv_heads, D,
                  bits=rng.choice([4, 4, 8]), group=rng.choice([32, 64, 128, 128]),
                  page=rng.choice([16, 32, 64, 128, 256]), dtype=rng.choice(["bf16", "f16"]), window=window,
                  sinks=rng.choice([0, 1, 4, 64]) if window else 0,
                  causal=True if window else rng.random() < 0.85)
        del c["name"]
        w = work(c)
        # several long prompts at once make large inputs: the rows a case holds are bounded too
        rows = sum(n + m for n, m in _lengths(c)) * kv_heads * D
        if all(w[k] <= most[kind, k] for k in ("bytes", "flops")) and rows <= 4 * 131072 * 8 * 128:
            return c


def _lengths(case):
    """(context, new) of every sequence, from the case alone."""
    return [(case["context"] - b * 7919 % (case["context_spread"] + 1), case["new"] - b * 37 % (case["new_spread"] + 1))
            for b in range(case["seqs"])]


def _row_bytes(case):
    return case["head_dim"] * case["bits"] // 8 + case["head_dim"] // case["group"] * 4


def work(case):
    D, Hk, Hq = case["head_dim"], case["kv_heads"], case["q_heads"]
    lens = _lengths(case)
    rows = sum(n for _, n in lens)
    if case["kind"] == "round":        # 16-bit rows in, codes written, 16-bit rows out
        return {"bytes": 2 * rows * Hk * (4 * D + _row_bytes(case)), "flops": 2 * rows * Hk * D * 8}
    if case["kind"] == "read":
        return {"bytes": 2 * rows * Hk * (2 * D + _row_bytes(case)), "flops": 2 * rows * Hk * D * 2}
    keys = pairs = 0
    for ctx, n in lens:
        total, w, s = ctx + n, case["window"], case["sinks"]
        if not case["causal"]:
            keys, pairs = keys + total, pairs + n * total
            continue
        first = max(0, ctx - w + 1) if w else 0          # first key the earliest row's window reaches
        keys += total - first + min(s, first)
        for i in ([0, n - 1] if not w else range(n)):
            p = ctx + i
            lo = max(0, p - w + 1) if w else 0
            vis = p + 1 - lo + min(s, lo)
            pairs += vis if w else (n / 2) * vis         # linear in i without a window
    return {"bytes": 2 * keys * Hk * _row_bytes(case) + 4 * rows * Hq * D, "flops": 4.0 * D * Hq * pairs}


# ---------------------------------------------------------------- inputs
def _draw_rows(case, seed, part, rows, what):
    """16-bit rows [rows, kv_heads, head_dim] of keys or values.  Keys have
    channels of very different size, as rotary keys do; values are even."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + part * 4 + (1 if what == "v" else 0))
    x = torch.randn(rows, case["kv_heads"], case["head_dim"], generator=g, device=DEV)
    if what == "k":
        gc = torch.Generator(device=DEV)
        gc.manual_seed(seed * 1000003 + 999999)
        x *= torch.exp(0.5 * torch.randn(case["kv_heads"], case["head_dim"], generator=gc, device=DEV))
    return x.to(DTYPES[case["dtype"]])


def _parts(case):
    """Runs of sequences whose cached rows are drawn together (about 2^17 rows at most, or one sequence)."""
    parts, now, rows = [], [], 0
    for b, (ctx, n) in enumerate(_lengths(case)):
        if now and rows + ctx + n > 1 << 17:
            parts.append(now)
            now, rows = [], 0
        now.append(b)
        rows += ctx + n
    return parts + [now]


def _table(case, seed):
    """Page table: every sequence's pages scattered over the cache; -1 behind its last page."""
    ps = case["page"]
    need = [(ctx + n + ps - 1) // ps for ctx, n in _lengths(case)]
    pages = sum(need) + 3
    g = torch.Generator()
    g.manual_seed(seed + 17)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((case["seqs"], max(need)), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table.to(DEV), pages


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _int32(v):
    return torch.tensor(v, dtype=torch.int32).to(DEV)


def prepare(case, seed):
    lens = _lengths(case)
    dtype, D = DTYPES[case["dtype"]], case["head_dim"]
    rows = sum(n for _, n in lens)
    table, pages = _table(case, seed)
    s = {"case": case, "lens": lens, "table": table, "rows": rows, "scale": D ** -0.5}
    if case["kind"] == "attend":
        g = torch.Generator(device=DEV)
        g.manual_seed(seed * 1000003 + 5)
        s["q"] = (1.5 * torch.randn(rows, case["q_heads"], D, generator=g, device=DEV)).to(dtype)
    if case["kind"] == "round":        # keys and values as slices of one projection's output
        s["kv"] = torch.stack([_draw_rows(case, seed, 7, rows, "k"), _draw_rows(case, seed, 7, rows, "v")], 1)

    if own:
        from error_compensated_bit_amd import binding as B
        cache = B.alloc_kv_cache(pages, case["page"], case["kv_heads"], D, bits=case["bits"], group=case["group"],
                                 device=DEV)
        new = [n for _, n in lens]
        batch = B.KVBatch(_int32(_starts(new)), _int32([c + n for c, n in lens]), table, rows=rows,
                          max_new=max(new), max_len=max(c + n for c, n in lens))
        s["cache"], s["batch"] = cache, batch
        if case["kind"] == "attend":
            s["out"] = torch.empty_like(s["q"])
            s["calls"] = [B.prepare_kv_attention(cache, batch, s["q"], s["out"], s["scale"], causal=case["causal"],
                                                 window=case["window"], sinks=case["sinks"])]
        else:
            s["k"] = torch.empty(rows, case["kv_heads"], D, dtype=dtype, device=DEV)
            s["v"] = torch.empty_like(s["k"])
            s["calls"] = [B.prepare_kv_read(cache, batch, s["k"], s["v"])]
            if case["kind"] == "round":
                s["calls"].insert(0, B.prepare_kv_write(cache, batch, s["kv"][:, 0], s["kv"][:, 1]))
    else:
        slots, groups = pages * case["page"], D // case["group"]
        for x in "kv":
            s[x + "_codes"] = torch.zeros(slots, case["kv_heads"], D, dtype=torch.uint8, device=DEV)
            s[x + "_step"] = torch.zeros(slots, case["kv_heads"], groups, dtype=torch.float16, device=DEV)
            s[x + "_zero"] = torch.zeros_like(s[x + "_step"])

    if case["kind"] != "round":        # the cache as earlier calls filled it
        for part, seqs in enumerate(_parts(case)):
            count = [lens[b][0] + lens[b][1] for b in seqs]
            k, v = (_draw_rows(case, seed, part, sum(count), x) for x in "kv")
            if own:
                B.echo_kv_write(cache, B.KVBatch(_int32(_starts(count)), _int32(count), table[seqs[0]:seqs[-1] + 1],
                                                 rows=sum(count), max_new=max(count), max_len=max(count)), k, v)
            else:
                at = torch.cat([_slots(case, table, b, 0, n) for b, n in zip(seqs, count)])
                _plain_write(s, at, k, v)
    return s


# ---------------------------------------------------------------- the plain form
def _slots(case, table, b, first, count):
    p = torch.arange(first, first + count, device=DEV)
    return table[b].long()[p // case["page"]] * case["page"] + p % case["page"]


def _plain_quantize(x, bits, group):
    """codes uint8 [..., D], step and zero fp16 [..., D / group] of rows x."""
    qmax = float(2 ** bits - 1)
    x = x.float().unflatten(-1, (-1, group))
    zero = x.amin(-1).clamp(-65504.0, 65504.0).half()
    zero = torch.where(zero == 0, torch.zeros_like(zero), zero)
    span = x.amax(-1) - zero.float()
    step = (span.double() / qmax).float()                  # a 64-bit quotient rounds to the binary32 one
    step = torch.where(step > 0, step.clamp(max=65504.0), torch.zeros_like(step)).half()
    inv = torch.where(step > 0, 1.0 / step.double(), torch.zeros_like(step, dtype=torch.float64)).float()
    code = ((x - zero.float()[..., None]) * inv[..., None]).round().clamp(0.0, qmax)
    return code.to(torch.uint8).flatten(-2), step, zero


def _plain_write(s, at, k, v):
    case = s["case"]
    for x, rows in (("k", k), ("v", v)):
        codes, step, zero = _plain_quantize(rows, case["bits"], case["group"])
        s[x + "_codes"][at] = codes
        s[x + "_step"][at] = step
        s[x + "_zero"][at] = zero


def _plain_values(s, x, at):
    """Dequantized fp32 rows [len(at), kv_heads, head_dim]: code * step is exact, the sum rounds once."""
    c = s[x + "_codes"][at].float().unflatten(-1, (-1, s["case"]["group"]))
    return (c * s[x + "_step"][at].float()[..., None] + s[x + "_zero"][at].float()[..., None]).flatten(-2)


def _plain_visible(case, ctx, n, total):
    p = torch.arange(ctx, ctx + n, device=DEV)[:, None]
    j = torch.arange(total, device=DEV)[None, :]
    if not case["causal"]:
        return torch.ones(n, total, dtype=torch.bool, device=DEV)
    vis = j <= p
    if case["window"]:
        vis = vis & ((p - j < case["window"]) | (j < case["sinks"]))
    return vis


def _plain_attend(s):
    case = s["case"]
    Hk, Hq, D = case["kv_heads"], case["q_heads"], case["head_dim"]
    r = Hq // Hk
    out = torch.empty_like(s["q"])
    first = 0
    for b, (ctx, n) in enumerate(s["lens"]):
        total = ctx + n
        at = _slots(case, s["table"], b, 0, total)
        k, v = (_plain_values(s, x, at) for x in "kv")
        q = s["q"][first:first + n].float()
        hidden = ~_plain_visible(case, ctx, n, total)
        for h in range(Hk):
            sc = torch.matmul(q[:, h * r:(h + 1) * r].reshape(n * r, D) * s["scale"], k[:, h].t().contiguous())
            sc = sc.view(n, r, total).masked_fill_(hidden[:, None, :], -math.inf)
            sc -= sc.amax(-1, keepdim=True)
            sc.exp_()
            o = torch.matmul(sc.view(n * r, total), v[:, h].contiguous()).view(n, r, D)
            out[first:first + n, h * r:(h + 1) * r] = (o / sc.sum(-1, keepdim=True)).to(out.dtype)
        first += n
    return out


def run(s):
    if own:
        for call in s["calls"]:
            call()
        return s["out"] if "out" in s else [s["k"], s["v"]]
    case = s["case"]
    if case["kind"] == "attend":
        return _plain_attend(s)
    at = torch.cat([_slots(case, s["table"], b, ctx, n) for b, (ctx, n) in enumerate(s["lens"])])
    if case["kind"] == "round":
        _plain_write(s, at, s["kv"][:, 0], s["kv"][:, 1])
    return [_plain_values(s, x, at).to(DTYPES[case["dtype"]]) for x in "kv"]


# ---------------------------------------------------------------- 64 bits
def _exact_values(x, bits, group):
    """Values (64 bits) that the cache holds for rows x, by the definition: every
    operation done in 64 bits and rounded to binary32 (or binary16) as it says."""
    def f32(t):
        return t.to(torch.float32).to(torch.float64)

    def f16(t):                       # by way of binary32, as the definition says
        return t.to(torch.float32).to(torch.float16).to(torch.float64)

    top = (1 << bits) - 1
    v = x.to(torch.float64).reshape(*x.shape[:-1], x.shape[-1] // group, group)
    low, high = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
    zero = f16(low.clamp(-65504, 65504))
    step = f16(f32(f32(high - zero) / top).clamp(0, 65504))
    inv = torch.where(step > 0, f32(1 / step), torch.zeros_like(step))
    code = torch.round(f32(f32(v - zero) * inv)).clamp(0, top)
    return (code * step + zero).reshape(x.shape)


def exact(case, seed):
    lens = _lengths(case)
    bits, group, D = case["bits"], case["group"], case["head_dim"]
    if case["kind"] == "round":
        rows = sum(n for _, n in lens)
        return [_exact_values(_draw_rows(case, seed, 7, rows, x), bits, group) for x in "kv"]
    if case["kind"] == "read":
        parts = [(p, sum(lens[b][1] for b in seqs)) for p, seqs in enumerate(_parts(case))]
        return [torch.cat([_exact_values(_draw_rows(case, seed, p, n, x), bits, group) for p, n in parts]) for x in "kv"]
    rows, Hq, Hk = sum(n for _, n in lens), case["q_heads"], case["kv_heads"]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 5)
    q = (1.5 * torch.randn(rows, Hq, D, generator=g, device=DEV)).to(DTYPES[case["dtype"]]).double()
    out = torch.empty(rows, Hq, D, dtype=torch.float64, device=DEV)
    first = 0
    for part, seqs in enumerate(_parts(case)):
        count = [sum(lens[b]) for b in seqs]
        ks, vs = (_draw_rows(case, seed, part, sum(count), x) for x in "kv")
        begin = 0
        for b, total in zip(seqs, count):
            ctx, n = lens[b]
            k, v = (_exact_values(t[begin:begin + total], bits, group) for t in (ks, vs))
            begin += total
            for i0 in range(0, n, 512):                   # query rows in pieces
                m = min(512, n - i0)
                far = torch.arange(ctx + i0, ctx + i0 + m, device=DEV).unsqueeze(1) - torch.arange(total, device=DEV)
                seen = torch.ones_like(far, dtype=torch.bool)
                if case["causal"]:
                    seen = far >= 0
                    if case["window"]:
                        seen &= (far < case["window"]) | (torch.arange(total, device=DEV) < case["sinks"])
                for h in range(Hq):
                    e = (q[first + i0:first + i0 + m, h] @ k[:, h * Hk // Hq].t().contiguous()) / math.sqrt(D)
                    w = torch.softmax(torch.where(seen, e, torch.full_like(e, -math.inf)), dim=1)
                    out[first + i0:first + i0 + m, h] = w @ v[:, h * Hk // Hq].contiguous()
            first += n
    return out
