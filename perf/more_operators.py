"""The operators around a decoder layer's quantized products, as cases for a benchmark: the RMS norm (with the
residual's addition) that hands its result on in 8 bits, the append of new keys and values to a paged cache
in 8 bits, and the attention that reads this cache, for single tokens and for prompts.

`run` computes a case with elementary torch operations in 32 bits (64 for the norm's sum of squares, which
decides between neighbouring codes), or through the library's own calls where `own` is set. `exact` computes
it in 64 bits from the definition, head by head.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"

EPS = 1e-6
MAXIMUM = {"fp8": 448.0, "int8": 127.0}     # of the codes
HEADS = (64, 96, 128, 192, 256)             # head sizes
PAGES = (16, 32, 64, 128, 256)              # tokens of a page


def listed():
    return [
        # one decoded token: residual added, normed, e4m3 with one scale for the next projection; latency counts
        {"name": "norm 1x4096 fp8", "op": "norm", "M": 1, "K": 4096, "fmt": "fp8", "residual": True, "both": False},
        # a decode batch in front of an MoE block: block-scaled e4m3 for the experts, bf16 for the router
        {"name": "norm 67x7168 block both", "op": "norm", "M": 67, "K": 7168, "fmt": "block", "residual": True, "both": True},
        # a prompt, INT8 with one scale a token
        {"name": "norm 8192x8192 int8", "op": "norm", "M": 8192, "K": 8192, "fmt": "int8", "residual": True, "both": False},
        # a prompt's first norm: no residual yet, MX blocks
        {"name": "norm 4099x5120 mxfp8", "op": "norm", "M": 4099, "K": 5120, "fmt": "mxfp8", "residual": False, "both": False},
        # a decode step's new tokens: one of each sequence, most into pages that hold others already
        {"name": "append 48x1 fp8", "op": "append", "fmt": "fp8", "B": 48, "new": 1, "ctx": 2000, "H": 8, "D": 128, "P": 16, "mix": 1},
        # prompts of different lengths packed behind each other
        {"name": "append 5 prompts int8", "op": "append", "fmt": "int8", "B": 5, "new": 4000, "ctx": 0, "H": 8, "D": 128, "P": 64, "mix": 2},
        # a short conversation, small heads, no sharing: the smallest call
        {"name": "attn 1x1 on 100", "op": "attn", "fmt": "fp8", "B": 1, "new": 1, "ctx": 100, "H": 8, "G": 1, "D": 64, "P": 16, "window": 0, "mix": 3},
        # one sequence with a long past: only the past can be split
        {"name": "attn 1x1 on 131071", "op": "attn", "fmt": "fp8", "B": 1, "new": 1, "ctx": 131071, "H": 8, "G": 4, "D": 128, "P": 64, "window": 0, "mix": 4},
        # a decode batch, ragged, eight query heads to a head of the cache
        {"name": "attn 64x1 on 8000 int8", "op": "attn", "fmt": "int8", "B": 64, "new": 1, "ctx": 8000, "H": 8, "G": 8, "D": 128, "P": 16, "window": 0, "mix": 5},
        # drafted tokens checked at once, a sliding window
        {"name": "attn 7x5 window 1024", "op": "attn", "fmt": "fp8", "B": 7, "new": 5, "ctx": 10000, "H": 4, "G": 6, "D": 256, "P": 32, "window": 1024, "mix": 6},
        # prompts packed behind each other
        {"name": "attn 4 prompts of 4500", "op": "attn", "fmt": "fp8", "B": 4, "new": 4500, "ctx": 0, "H": 8, "G": 4, "D": 128, "P": 64, "window": 0, "mix": 7},
        # a prompt taken in pieces: the piece against everything before it
        {"name": "attn 1x1024 on 30000 int8", "op": "attn", "fmt": "int8", "B": 1, "new": 1024, "ctx": 30000, "H": 8, "G": 8, "D": 128, "P": 128, "window": 0, "mix": 8},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("norm", "append", "attn", "attn"))
    if op == "norm":
        fmt = rng.choice(("bf16", "fp8", "int8", "block", "mxfp8"))
        unit = {"block": 128, "mxfp8": 32}.get(fmt, 8)
        K = unit * _log(rng, max(1, 64 // unit), 16384 // unit)
        return {"op": "norm", "M": _log(rng, 1, min(16384, 60_000_000 // K)), "K": K, "fmt": fmt, "residual": rng.random() < 0.7,
                "both": fmt != "bf16" and rng.random() < 0.3}
    c = {"op": op, "fmt": rng.choice(("fp8", "int8")), "H": _log(rng, 1, 16), "D": rng.choice(HEADS), "P": rng.choice(PAGES), "mix": rng.randrange(1 << 30)}
    if op == "append":
        new = rng.choice((1, _log(rng, 2, 16), _log(rng, 17, 8192)))
        B = _log(rng, 1, min(256, max(1, 30_000_000 // (new * c["H"] * c["D"]))))
        return {**c, "B": B, "new": new, "ctx": rng.choice((0, _log(rng, 1, 4000)))}
    c["G"] = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 16))
    c["window"] = rng.choice((0, 0, 0, _log(rng, 16, 8192)))
    if rng.random() < 0.65:
        new = rng.choice((1, 1, rng.randint(2, 16)))
        ctx = _log(rng, 16, 131072)
        B = _log(rng, 1, max(1, min(128, 400_000_000 // (ctx * c["H"] * c["D"]))))
    else:
        new = _log(rng, 17, 4096)
        ctx = rng.choice((0, _log(rng, 16, 16384)))
        most = 230_000_000_000 // (new * (new + ctx) * c["D"])      # query heads, over all sequences
        c["H"] = max(1, min(c["H"], most // c["G"]))
        B = _log(rng, 1, max(1, min(16, most // (c["H"] * c["G"]))))
    return {**c, "B": B, "new": new, "ctx": ctx}


# ---- inputs -----------------------------------------------------------------------------------


def _lens(c):
    """New tokens and length after them, of each sequence: the first takes the largest of both, the others down to a
    quarter of that."""
    r = random.Random(c["mix"])
    some = lambda most: most - r.randint(0, most * 3 // 4)  # noqa: E731
    new = [c["new"]] + [max(1, some(c["new"])) for _ in range(c["B"] - 1)]
    return new, [n + p for n, p in zip(new, [c["ctx"]] + [some(c["ctx"]) for _ in range(c["B"] - 1)])]


def _tables(c, g):
    """The pages of each sequence, in no order, -1 behind its last one; and how many there are."""
    _, lens = _lens(c)
    held = [-(-n // c["P"]) for n in lens]
    order = torch.randperm(sum(held), generator=g, device=DEV).to(torch.int32).cpu()
    table, at = torch.full((c["B"], max(held)), -1, dtype=torch.int32), 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(held)


def _cache(c, g, pages, what):
    """Pages of a cache that is in use: values about N(0, 1) (keys with some channels several times as large) quantized
    page by page, so that every page's largest code is the type's largest."""
    x = torch.randn((pages, c["H"], c["P"], c["D"]), generator=g, device=DEV)
    if what == "k":
        x *= 1 + 4 * (torch.rand((c["H"], 1, c["D"]), generator=g, device=DEV) < 0.03)
    s = x.abs().amax((2, 3)) / MAXIMUM[c["fmt"]]
    x /= s[:, :, None, None]
    x = x.to(torch.float8_e4m3fn).view(torch.uint8) if c["fmt"] == "fp8" else x.round_().to(torch.int8).view(torch.uint8)
    return (x if what == "k" else x.transpose(2, 3)).contiguous(), s


def _made(case, seed):
    """The inputs, from the seed alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = case
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        size = 0.5 + torch.rand((M, 1), generator=g, device=DEV)
        x = (size * torch.randn((M, K), generator=g, device=DEV)).to(torch.bfloat16)
        r = None
        if c["residual"]:   # the stream: a few channels far larger than the others
            r = torch.randn((M, K), generator=g, device=DEV) * (1 + 20 * (torch.rand(K, generator=g, device=DEV) < 0.002))
            r = r.to(torch.bfloat16)
        return {"x": x, "residual": r, "weight": (0.5 + torch.rand(K, generator=g, device=DEV)).to(torch.bfloat16)}
    new, lens = _lens(c)
    table, pages = _tables(c, g)
    T, H, D = sum(new), c["H"], c["D"]
    m = {"cu": torch.tensor([sum(new[:b]) for b in range(c["B"] + 1)], dtype=torch.int32, device=DEV),
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "table": table.to(DEV)}
    m["k_pages"], m["k_scales"] = _cache(c, g, pages, "k")
    m["v_pages"], m["v_scales"] = _cache(c, g, pages, "v")
    # what the projection of queries, keys and values leaves: all heads of a token in one row
    Hq = H * c.get("G", 1)
    qkv = torch.randn((T, Hq + 2 * H, D), generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = qkv.split((Hq, H, H), 1)
    return {**m, "q": q} if c["op"] == "attn" else {**m, "k": k, "v": v}


def _desc(hq, c, pages):
    return hq.make_kv_desc(hq.HQ_KV_FP8_E4M3 if c["fmt"] == "fp8" else hq.HQ_KV_INT8, c["H"], c["D"], c["P"], pages)


def prepare(case, seed):
    c = case
    s = {"case": dict(c), **_made(c, seed)}
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        # what a program holds for a norm's results
        s["y"] = torch.empty((M, K), dtype=torch.bfloat16 if c["fmt"] == "bf16" else torch.uint8, device=DEV)
        s["scale"] = {"bf16": None, "block": torch.empty((M, K // 128), device=DEV), "mxfp8": torch.empty((M, K // 32), dtype=torch.uint8, device=DEV)}.get(
            c["fmt"], torch.empty(M, device=DEV))
        s["copy"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV) if c["both"] else None
        s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
    elif c["op"] == "append":
        # where each touched page's new tokens come from (-1: no new one there), as a scheduler that hands out the pages knows it
        new, lens = _lens(c)
        table, P = s["table"].cpu(), c["P"]
        pages, rows, at = [], [], 0
        for b, (n, end) in enumerate(zip(new, lens)):
            for p in range((end - n) // P, -(-end // P)):
                pages.append(int(table[b, p]))
                rows.append([at + p * P + i - (end - n) if end - n <= p * P + i < end else -1 for i in range(P)])
            at += n
        s["touched"] = torch.tensor(pages, device=DEV)
        s["rows"] = torch.tensor(rows, device=DEV)
    else:
        s["out"] = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    if own:
        import quantized_gemm_prepacked_amd as hq
        s["hq"] = hq
        if c["op"] == "norm":
            s["fmt"] = {"bf16": hq.HQ_ACT_BF16, "fp8": hq.HQ_ACT_FP8E4M3_PER_TOKEN, "int8": hq.HQ_ACT_INT8_PER_TOKEN,
                        "block": hq.HQ_ACT_FP8E4M3_BLOCK128, "mxfp8": hq.HQ_ACT_MXFP8}[c["fmt"]]
        else:
            s["desc"] = _desc(hq, c, s["k_pages"].shape[0])
        if c["op"] == "attn":
            s["longest"] = max(_lens(c)[1])
            s["ws_bytes"] = hq.hq_attention_workspace_bytes(s["desc"], c["B"], s["q"].shape[0], c["H"] * c["G"], c["new"], s["longest"])
            s["ws"] = torch.empty(max(1, s["ws_bytes"]), dtype=torch.uint8, device=DEV)
    return s


# ---- the plain forms --------------------------------------------------------------------------


def _coded(x, fmt):
    """The codes' values of x, which is already divided by its scale."""
    if fmt == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _norm(s, c):
    h = s["x"].float()
    if c["residual"]:
        h = (h + s["residual"].float()).to(torch.bfloat16)
        out = {"sum": h}
        h = h.float()
    else:
        out = {}
    inv = (1 / (h.double().square().sum(1, keepdim=True) / c["K"] + EPS).sqrt()).float()
    y = h * inv * s["weight"].float()
    if c["fmt"] == "bf16":
        return {**out, "y": y.to(torch.bfloat16)}
    if c["both"]:
        out["copy"] = y.to(torch.bfloat16)
    if c["fmt"] == "mxfp8":
        y = y.unflatten(1, (-1, 32))
        top = y.abs().amax(2)
        e = torch.where(top > 0, torch.frexp(top).exponent - 9, -127).clamp(-127, 127)
        code = _coded(torch.ldexp(y, -e[..., None]), "fp8")
        return {**out, "y": code.flatten(1), "scale": (e + 127).to(torch.uint8)}
    if c["fmt"] == "block":
        y = y.unflatten(1, (-1, 128))
    scale = y.abs().amax(-1, keepdim=True) / MAXIMUM["int8" if c["fmt"] == "int8" else "fp8"]
    scale = torch.where(scale == 0, 1.0, scale)
    code = _coded(y / scale, "int8" if c["fmt"] == "int8" else "fp8")
    return {**out, "y": code.reshape(c["M"], c["K"]), "scale": scale.squeeze(-1)}


def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "fp8" else torch.int8)


def _append(s, c, what):
    """One of the two caches, its touched pages written anew."""
    fmt, rows, pages, scales = c["fmt"], s["rows"], s[what + "_pages"], s[what + "_scales"]
    is_new = (rows >= 0)[:, :, None, None]
    is_old = (rows.cummax(1).values < 0)[:, None, :, None]      # slots before the first new one
    x = torch.where(is_new, s[what][rows.clamp_min(0)].float(), 0.0).transpose(1, 2)     # [touched, H, P, D]
    need, held = x.abs().amax((2, 3)) / MAXIMUM[fmt], scales[s["touched"]]
    held = torch.where(((rows[:, :1] >= 0) | (held == 0)), need, held)
    # the smallest power of two by which the held scale has to grow
    (mn, en), (mh, eh) = torch.frexp(need), torch.frexp(held)
    grow = torch.where(need > held, en - eh + (mn > mh), 0)
    scale = torch.ldexp(held, grow)
    old = pages[s["touched"]]
    old = old if what == "k" else old.transpose(2, 3)
    moved = _coded(torch.ldexp(_values(old, fmt).float(), -grow[:, :, None, None]), fmt).view(torch.uint8)
    code = _coded(x / torch.where(scale == 0, 1.0, scale)[:, :, None, None], fmt).view(torch.uint8)
    code = torch.where(is_new.transpose(1, 2), code, torch.where(is_old, moved, old))
    pages[s["touched"]] = code if what == "k" else code.transpose(2, 3)
    scales[s["touched"]] = scale


def _gathered(s, c, what):
    """The cache of every sequence as values, [B, H, tokens, D], zeros where the table has no page."""
    table = s["table"].long()
    x = s[what + "_pages"][table.clamp_min(0)]                               # [B, pages, H, P, D] (v: D, P)
    x = _values(x if what == "k" else x.transpose(3, 4).contiguous(), c["fmt"]).float()
    x = x * torch.where(table[:, :, None] >= 0, s[what + "_scales"][table.clamp_min(0)], 0.0)[..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend(s, c):
    H, G, n = c["H"], c["G"], c["new"]
    first, count = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(n, device=DEV)
    live = i < count[:, None]                                                # [B, n]
    row = torch.where(live, first[:, None] + i, 0)
    q = s["q"][row].float().unflatten(2, (H, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)       # [B, H, G * n, D]
    score = torch.matmul(q, _gathered(s, c, "k").transpose(2, 3).contiguous()) * c["D"] ** -0.5
    at = (s["lens"].long() - count)[:, None] + i                             # [B, n]: each query's position
    j = torch.arange(score.shape[3], device=DEV)
    seen = (j <= at[..., None]) & live[..., None]
    if c["window"]:
        seen &= j > at[..., None] - c["window"]
    score = score.unflatten(2, (G, n)).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), _gathered(s, c, "v")).unflatten(2, (G, n)) / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[live].to(torch.bfloat16)   # rows in the packed order


def run(state):
    s, c = state, state["case"]
    if own:
        hq = s["hq"]
        if c["op"] == "norm":
            hq.hq_rms_norm(s["fmt"], c["M"], c["K"], s["x"], s["residual"], s["weight"], EPS, s["sum"], s["y"], s["scale"], s["copy"])
            out = {"y": s["y"] if c["fmt"] == "bf16" else s["y"].view(torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn)}
            for name in ("sum", "copy", "scale"):
                if s[name] is not None:
                    out[name] = s[name]
            return out
        if c["op"] == "append":
            hq.hq_kv_append(s["desc"], c["B"], s["k"].shape[0], c["new"], s["k"], s["v"], s["k"].stride(0), s["cu"], s["lens"], s["table"],
                            s["table"].shape[1], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        else:
            hq.hq_attention(s["desc"], c["B"], s["q"].shape[0], c["H"] * c["G"], c["new"], s["longest"], s["q"], s["q"].stride(0), s["cu"], s["lens"],
                            s["table"], s["table"].shape[1], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], c["D"] ** -0.5, c["window"],
                            s["out"], s["ws"], s["ws_bytes"])
            return s["out"]
    elif c["op"] == "norm":
        return _norm(s, c)
    elif c["op"] == "attn":
        return _attend(s, c)
    else:
        _append(s, c, "k")
        _append(s, c, "v")
    return {"k": _values(s["k_pages"], c["fmt"]), "v": _values(s["v_pages"], c["fmt"]), "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


# ---- the definitions in 64 bits ---------------------------------------------------------------


def _round64(x, fmt):
    """The nearest value that a code can hold, ties to the even code."""
    if fmt == "int8":
        return torch.round(x.clamp(-127, 127))
    x = x.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _decoded64(codes, fmt):
    v = codes.to(torch.int64)
    if fmt == "int8":
        return (v - 256 * (v > 127)).double()
    mant, exp = (v & 7).double(), (v >> 3 & 15).double()
    return torch.where(exp == 0, mant * 2.0 ** -9, (8 + mant) * torch.exp2(exp - 10)) * (1 - 2 * (v > 127).double())


def _exact_norm(c, m):
    h, out = m["x"].double(), {}
    if c["residual"]:
        h = h + m["residual"].double()
        out["sum"] = h
        h = h.to(torch.bfloat16).double()       # the stream is held in bf16, and that is what is normed
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * m["weight"].double()
    if c["fmt"] == "bf16":
        return {**out, "y": y}
    if c["both"]:
        out["copy"] = y
    if c["fmt"] == "mxfp8":
        y = y.view(c["M"], -1, 32)
        e = torch.floor(torch.log2(y.abs().amax(2))) - 8
        return {**out, "y": _round64(y * torch.exp2(-e)[..., None], "fp8").view(c["M"], -1), "scale": (e + 127).to(torch.uint8)}
    kind = "int8" if c["fmt"] == "int8" else "fp8"
    y = y.view(c["M"], -1, 128 if c["fmt"] == "block" else c["K"])
    scale = y.abs().amax(2) / MAXIMUM[kind]
    code = _round64(y / scale[..., None], kind).view(c["M"], -1)
    return {**out, "y": code.to(torch.int8) if kind == "int8" else code, "scale": scale.view(c["M"], -1) if c["fmt"] == "block" else scale[:, 0]}


def _exact_append(c, m):
    fmt, P = c["fmt"], c["P"]
    new, lens = _lens(c)
    table, cu = m["table"].tolist(), m["cu"].tolist()
    out = {}
    for what in ("k", "v"):
        codes = _decoded64(m[what + "_pages"], fmt)
        codes = codes if what == "k" else codes.transpose(2, 3)
        scales, x = m[what + "_scales"].double(), m[what].double()
        for b, (n, end) in enumerate(zip(new, lens)):
            begin = end - n
            for p in range(begin // P, -(-end // P)):
                page, lo, hi = table[b][p], max(begin, p * P), min(end, (p + 1) * P)
                part = x[cu[b] + lo - begin:cu[b] + hi - begin].transpose(0, 1)          # [H, tokens, D]
                need = part.abs().amax((1, 2)) / MAXIMUM[fmt]
                # scales are held in 32 bits, and the codes go by what is held
                need = need.float().double()
                if lo == p * P:
                    scale = need
                else:
                    # (every value of a cache in use is from the middle of its type's range: no scale of zero)
                    scale = scales[page]
                    grow = torch.exp2(torch.ceil(torch.log2(need / scale)).clamp_min(0))
                    codes[page, :, :lo - p * P] = _round64(codes[page, :, :lo - p * P] / grow[:, None, None], fmt)
                    scale = scale * grow
                codes[page, :, lo - p * P:hi - p * P] = _round64(part / scale[:, None, None], fmt)
                scales[page] = scale
        codes = codes if what == "k" else codes.transpose(2, 3)
        out[what], out[what + "_scales"] = codes.to(torch.int8) if fmt == "int8" else codes, scales
    return out


def _exact_attend(c, m):
    fmt, G, P, H = c["fmt"], c["G"], c["P"], c["H"]
    new, lens = _lens(c)
    cu = m["cu"].tolist()
    out = torch.zeros(m["q"].shape, dtype=torch.float64, device=DEV)
    for b, (n, end) in enumerate(zip(new, lens)):
        pages = m["table"][b, :-(-end // P)].long()
        at = torch.arange(end - n, end, device=DEV)[:, None]
        j = torch.arange(end, device=DEV)[None]
        hidden = j > at
        if c["window"]:
            hidden |= j <= at - c["window"]
        for h in range(H):
            k = (_decoded64(m["k_pages"][pages, h], fmt) * m["k_scales"][pages, h].double()[:, None, None]).reshape(-1, c["D"])[:end]
            v = _decoded64(m["v_pages"][pages, h], fmt) * m["v_scales"][pages, h].double()[:, None, None]
            v = v.transpose(1, 2).reshape(-1, c["D"])[:end]
            for i in range(h * G, h * G + G):
                score = m["q"][cu[b]:cu[b + 1], i].double() @ k.T / math.sqrt(c["D"])
                out[cu[b]:cu[b + 1], i] = torch.softmax(score.masked_fill_(hidden, -math.inf), 1) @ v
    return out


def exact(case, seed):
    c, m = case, _made(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attn": _exact_attend}[c["op"]](c, m)


# ---- what a case cannot do without ------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        out = {"bf16": 2 * K, "fp8": K + 4, "int8": K + 4, "block": K + K / 32, "mxfp8": K + K / 32}[c["fmt"]]
        return {"bytes": M * (2 * K + (4 * K if c["residual"] else 0) + out + (2 * K if c["both"] else 0)) + 2 * K, "flops": 8 * M * K}
    new, lens = _lens(c)
    H, D, P = c["H"], c["D"], c["P"]
    if c["op"] == "append":
        touched = sum(-(-end // P) - (end - n) // P for n, end in zip(new, lens))
        return {"bytes": sum(new) * H * D * 6 + touched * (16 * H + 4), "flops": 8 * sum(new) * H * D}
    read, products = 0, 0
    for n, end in zip(new, lens):
        w = c["window"] or end
        read += end - max(0, end - n - w + 1)
        products += sum(min(w, p + 1) for p in range(end - n, end)) if c["window"] else n * (2 * end - n + 1) // 2
    return {"bytes": read * H * (2 * D + 8 / P) + sum(new) * H * c["G"] * D * 4, "flops": 4 * D * H * c["G"] * products}
