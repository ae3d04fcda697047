"""The decode-step operators, as cases for a benchmark: the MoE router's selection, matrix-vector
products with packed weights (plain and gated), and the MoE layer for a few tokens.

`run` computes a case with elementary torch operations in 32 bits (64 for the router's selection
values, which decide between neighbours), or through the library's own calls where `own` is set.
`exact` computes it in 64 bits, expert by expert, from the definition.
"""
import math

import torch

own = False

DEV = "cuda:0"

# e2m1 magnitudes by code (the fourth bit is the sign)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decoded token of a model with 256 experts: the router is a single row, latency counts
        {"name": "route 1x256 top8", "op": "route", "T": 1, "E": 256, "topk": 8, "bf16": False, "sigmoid": False,
         "bias": False, "groups": 1, "keep": 1, "renorm": True, "masked": 0.0},
        # a decode batch on bf16 logits (real ties), no renormalisation, some experts switched off
        {"name": "route 67x60 top4 bf16", "op": "route", "T": 67, "E": 60, "topk": 4, "bf16": True, "sigmoid": False,
         "bias": False, "groups": 1, "keep": 1, "renorm": False, "masked": 0.1},
        # prefill: sigmoid scores with a balancing bias, the best 4 of 8 expert groups
        {"name": "route 4096x256 groups", "op": "route", "T": 4096, "E": 256, "topk": 8, "bf16": False,
         "sigmoid": True, "bias": True, "groups": 8, "keep": 4, "renorm": True, "masked": 0.0},
        # the tiny projection: nothing but latency
        {"name": "gemv 1x256x512 int4 g32", "op": "gemv", "M": 1, "N": 256, "K": 512, "fmt": "int4", "group": 32, "gated": False},
        # one token through a wide projection at the dense sweep's shape
        {"name": "gemv 1x14336x4096 uint4 g64", "op": "gemv", "M": 1, "N": 14336, "K": 4096, "fmt": "uint4", "group": 64, "gated": False},
        # three sequences through the gate and up projections of a dense gated MLP
        {"name": "gated 3x2x14336x4096 int4 g32", "op": "gemv", "M": 3, "N": 28672, "K": 4096, "fmt": "int4", "group": 32, "gated": True},
        # a decode batch of 13 (odd) on a square layer with an odd number of channel tiles
        {"name": "gemv 13x8208x8192 uint4 g128", "op": "gemv", "M": 13, "N": 8208, "K": 8192, "fmt": "uint4", "group": 128, "gated": False},
        # one decoded token, large experts
        {"name": "moe 1 7168x2048 int4 g128", "op": "moe", "T": 1, "topk": 8, "E": 32, "H": 7168, "I": 2048, "fmt": "int4", "group": 128},
        # one decoded token, many small MXFP4 experts: latency and few bytes
        {"name": "moe 1 2048x768 mxfp4", "op": "moe", "T": 1, "topk": 8, "E": 64, "H": 2048, "I": 768, "fmt": "mxfp4", "group": 32},
        # three sequences, asymmetric weights with fine groups
        {"name": "moe 3 4096x1408 uint4 g64", "op": "moe", "T": 3, "topk": 6, "E": 40, "H": 4096, "I": 1408, "fmt": "uint4", "group": 64},
        # a full decode batch: most experts are hit, several tokens share one
        {"name": "moe 16 4096x1536 int4 g32", "op": "moe", "T": 16, "topk": 4, "E": 64, "H": 4096, "I": 1536, "fmt": "int4", "group": 32},
        # 8-bit experts, a small batch
        {"name": "moe 4 2048x1024 fp8", "op": "moe", "T": 4, "topk": 2, "E": 16, "H": 2048, "I": 1024, "fmt": "fp8", "group": 0},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("route", "gemv", "gemv", "moe", "moe"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        keep = rng.randint(1, groups)
        return {"op": "route", "T": _log(rng, 1, 16384), "E": E, "topk": rng.randint(1, min(16, E // groups * keep)),
                "bf16": rng.random() < 0.5, "sigmoid": rng.random() < 0.5, "bias": rng.random() < 0.5, "groups": groups,
                "keep": keep, "renorm": rng.random() < 0.5, "masked": rng.choice((0.0, 0.0, 0.05, 0.5))}
    fmt, group = rng.choice((("int4", 32), ("int4", 64), ("int4", 128), ("uint4", 32), ("uint4", 64), ("uint4", 128),
                             ("mxfp4", 32), ("int8", 0), ("fp8", 0)))
    if op == "gemv":
        gated = rng.random() < 0.4
        K = 128 * _log(rng, 1, 128)
        most = 50_000_000 // K // 16
        N = 16 * _log(rng, 1, min(1792, most)) * (2 if gated else 1)
        return {"op": "gemv", "M": _log(rng, 1, 16), "N": N, "K": K, "fmt": fmt, "group": group, "gated": gated}
    H, I = 128 * _log(rng, 2, 56), 128 * _log(rng, 1, 16)
    E = max(4, min(_log(rng, 4, 128), (700_000_000 if "4" in fmt else 350_000_000) // (3 * H * I)))
    return {"op": "moe", "T": _log(rng, 1, 16), "topk": rng.randint(1, min(8, E)), "E": E, "H": H, "I": I, "fmt": fmt, "group": group}


# ---- inputs -----------------------------------------------------------------------------------


def _weights(g, E, N, K, fmt, group):
    """Quantized weights in the standard format: codes, scales and (uint4) zero-points, values about
    N(0, 1/K), as quantizing a trained layer leaves them."""
    std = K ** -0.5
    w = {"codes": torch.empty((E, N, K // 2 if "4" in fmt else K), dtype=torch.uint8, device=DEV), "zeros": None}
    for e in range(E):
        r = torch.randn((N, K), generator=g, device=DEV, dtype=torch.float16)
        if fmt == "int8":
            w["codes"][e] = (r * 32).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
        elif fmt == "fp8":
            w["codes"][e] = (r * 64).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            if fmt == "mxfp4":
                c = torch.bucketize(r.abs() * 1.5, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV, dtype=torch.float16))
                c = (c + 8 * (r < 0)).to(torch.uint8)
            elif fmt == "int4":
                c = ((r * 2.5).round().clamp(-8, 7).to(torch.int8) & 15).to(torch.uint8)
            else:
                c = (r * 2.5 + 7.5).round().clamp(0, 15).to(torch.uint8)
            w["codes"][e] = c[:, 0::2] | (c[:, 1::2] << 4)
    if fmt in ("int8", "fp8"):
        w["scales"] = std / (32 if fmt == "int8" else 64) * (0.7 + 0.6 * torch.rand((E, N), generator=g, device=DEV))
    elif fmt == "mxfp4":
        at = 127 + round(math.log2(std / 1.5))
        w["scales"] = torch.randint(at - 1, at + 2, (E, N, K // 32), generator=g, device=DEV).to(torch.uint8)
    else:
        w["scales"] = (std / 2.5 * (0.7 + 0.6 * torch.rand((E, N, K // group), generator=g, device=DEV))).to(torch.bfloat16)
        if fmt == "uint4":
            w["zeros"] = torch.randint(5, 11, (E, N, K // group), generator=g, device=DEV).to(torch.uint8)
    return w


def _made(case, seed):
    """The inputs, from the seed alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = case
    if c["op"] == "route":
        logits = 1.5 * torch.randn((c["T"], c["E"]), generator=g, device=DEV)
        off = torch.rand(c["E"], generator=g, device=DEV) < c["masked"]
        logits = torch.where(off, -math.inf, logits).to(torch.bfloat16 if c["bf16"] else torch.float32)
        bias = 0.05 * torch.randn(c["E"], generator=g, device=DEV) if c["bias"] else None
        return {"logits": logits, "bias": bias}
    if c["op"] == "gemv":
        x = torch.randn((c["M"], c["K"]), generator=g, device=DEV).to(torch.bfloat16)
        return {"x": x, "w": _weights(g, 1, c["N"], c["K"], c["fmt"], c["group"])}
    T, E, k = c["T"], c["E"], c["topk"]
    x = torch.randn((T, c["H"]), generator=g, device=DEV).to(torch.bfloat16)
    top = torch.softmax(torch.randn((T, E), generator=g, device=DEV), 1).topk(k, 1)
    return {"x": x, "ids": top.indices.to(torch.int32), "weights": top.values / top.values.sum(1, keepdim=True),
            "gate_up": _weights(g, E, 2 * c["I"], c["H"], c["fmt"], c["group"]),
            "down": _weights(g, E, c["H"], c["I"], c["fmt"], c["group"])}


def _desc(hq, fmt, group):
    if fmt in ("int4", "uint4"):
        a = fmt == "uint4"
        return hq.make_desc(hq.HQ_W_UINT4_ASYM if a else hq.HQ_W_INT4_SYM, group, hq.HQ_SCALE_BF16, int(a), hq.HQ_ACT_BF16)
    return {"mxfp4": hq.DESC_W4A16_MXFP4, "int8": hq.DESC_W8A16_INT8, "fp8": hq.DESC_W8A16_FP8}[fmt]


def _packed(hq, desc, w, N, K):
    """The weights in the kernels' layout, as a program does once when it loads a layer."""
    import numpy as np
    host = {k: v if v is None else (v.view(torch.int16) if v.dtype == torch.bfloat16 else v).cpu().numpy() for k, v in w.items()}
    E = host["codes"].shape[0]
    out = np.empty(hq.hq_decode_prepacked_bytes(desc, E, N, K), np.uint8)
    hq.hq_decode_prepack_weights(desc, E, N, K, host["codes"], host["scales"], host["zeros"], out)
    return torch.from_numpy(out).to(DEV)


def prepare(case, seed):
    c = case
    s = {"case": dict(c), **_made(c, seed)}
    if own:
        # what a program that uses the library holds: packed weights, outputs and a workspace
        import quantized_gemm_prepacked_amd as hq
        s["hq"] = hq
        if c["op"] == "route":
            s["ids"] = torch.empty((c["T"], c["topk"]), dtype=torch.int32, device=DEV)
            s["weights"] = torch.empty((c["T"], c["topk"]), dtype=torch.float32, device=DEV)
        elif c["op"] == "gemv":
            s["desc"] = _desc(hq, c["fmt"], c["group"])
            s["packed"] = _packed(hq, s["desc"], s.pop("w"), c["N"], c["K"])
            s["y"] = torch.empty((c["M"], c["N"] // (2 if c["gated"] else 1)), dtype=torch.bfloat16, device=DEV)
        else:
            s["desc"] = d = _desc(hq, c["fmt"], c["group"])
            s["gate_up"] = _packed(hq, d, s["gate_up"], 2 * c["I"], c["H"])
            s["down"] = _packed(hq, d, s["down"], c["H"], c["I"])
            s["out"] = torch.empty((c["T"], c["H"]), dtype=torch.bfloat16, device=DEV)
            s["ws_bytes"] = hq.hq_moe_decode_workspace_bytes(d, c["T"], c["topk"], c["E"], c["H"], c["I"])
            s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
    return s


# ---- the plain forms --------------------------------------------------------------------------


def _dequantized(w, fmt):
    """[E, N, K] in 32 bits (each value is exact there)."""
    codes, scales = w["codes"], w["scales"]
    if fmt == "int8":
        return codes.view(torch.int8).float() * scales[..., None]
    if fmt == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * scales[..., None]
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    q = q.unflatten(-1, (scales.shape[-1], -1))
    if fmt == "mxfp4":
        values = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        v = values[q.int()] * torch.exp2(scales.float() - 127)[..., None]
    elif fmt == "int4":
        v = ((q ^ 8).float() - 8) * scales.float()[..., None]
    else:
        v = (q.float() - w["zeros"].float()[..., None]) * scales.float()[..., None]
    return v.flatten(-2)


def _silu_mul(gu):
    g, u = gu.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def _route(s, c):
    l = s["logits"].double()
    l = torch.where(torch.isnan(l), -math.inf, l)
    if c["sigmoid"]:
        score = 1 / (1 + torch.exp(-l))
    else:
        top = l.max(1, keepdim=True).values
        e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
        score = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    value = score if s["bias"] is None else score + s["bias"].double()
    value = torch.where(l == -math.inf, -math.inf, value)
    by = l if s["bias"] is None else value
    if c["groups"] > 1:
        per = value.unflatten(1, (c["groups"], -1))
        two = per.sort(dim=2, descending=True).values[..., :2]
        best = torch.where(two == -math.inf, 0.0, two).sum(2)
        best = torch.where(two[..., 0] == -math.inf, -math.inf, best)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        stays = torch.zeros_like(best).scatter(1, kept, 1.0) > 0
        by = torch.where(stays.repeat_interleave(per.shape[2], 1), by, -math.inf)
    order = by.sort(dim=1, descending=True, stable=True)
    ids, gone = order.indices[:, : c["topk"]], order.values[:, : c["topk"]] == -math.inf
    w = torch.where(gone, 0.0, score.gather(1, ids))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"ids": torch.where(gone, -1, ids).int(), "weights": (w * SCALE).float()}


#: the factor on the router's weights
SCALE = 2.5


def run(state):
    s, c = state, state["case"]
    if own:
        hq = s["hq"]
        if c["op"] == "route":
            hq.hq_moe_route(hq.HQ_SCORE_SIGMOID if c["sigmoid"] else hq.HQ_SCORE_SOFTMAX, c["T"], c["E"], c["topk"], s["logits"],
                            hq.HQ_LOGITS_BF16 if c["bf16"] else hq.HQ_LOGITS_FP32, s["bias"], c["groups"], c["keep"], 2,
                            c["renorm"], SCALE, s["ids"], s["weights"])
            return {"ids": s["ids"], "weights": s["weights"]}
        if c["op"] == "gemv":
            hq.hq_gemv(s["desc"], hq.HQ_GEMV_SILU_MUL if c["gated"] else hq.HQ_GEMV_LINEAR, c["M"], c["N"], c["K"], s["x"],
                       s["packed"], s["y"])
            return s["y"]
        hq.hq_moe_decode(s["desc"], c["T"], c["topk"], c["E"], c["H"], c["I"], s["x"], s["ids"], s["weights"], s["gate_up"],
                         s["down"], s["out"], s["ws"], s["ws_bytes"])
        return s["out"]
    if c["op"] == "route":
        return _route(s, c)
    if c["op"] == "gemv":
        y = s["x"].float() @ _dequantized(s["w"], c["fmt"])[0].T
        return (_silu_mul(y) if c["gated"] else y).to(torch.bfloat16)
    # the experts that are used, each once: dequantized, applied to every token, the routed ones kept
    T, k = c["T"], c["topk"]
    used, at = torch.unique(s["ids"], return_inverse=True)
    used, token = used.long(), torch.arange(T, device=DEV)[:, None]
    part = lambda w: {n: None if v is None else v.view(torch.uint8)[used].view(v.dtype) for n, v in w.items()}  # noqa: E731
    gate_up = _dequantized(part(s["gate_up"]), c["fmt"])
    act = _silu_mul((s["x"].float() @ gate_up.flatten(0, 1).T).unflatten(1, (len(used), -1))[token, at.view(T, k)])
    del gate_up
    share = torch.zeros((T, len(used), c["I"]), device=DEV)
    share[token, at.view(T, k)] = act * s["weights"][..., None]
    down = _dequantized(part(s["down"]), c["fmt"])
    return torch.bmm(share.transpose(0, 1).contiguous(), down.transpose(1, 2).contiguous()).sum(0).to(torch.bfloat16)


# ---- the definitions in 64 bits ---------------------------------------------------------------


def _expert64(w, e, fmt, group):
    codes = w["codes"][e]
    if fmt in ("int8", "fp8"):
        v = codes.to(torch.int64)
        if fmt == "int8":
            v = (v - 256 * (v > 127)).double()
        else:
            mant, exp = (v & 7).double(), (v >> 3 & 15).double()
            v = torch.where(exp == 0, mant * 2.0 ** -9, (8 + mant) * torch.exp2(exp - 10)) * (1 - 2 * (v > 127).double())
        return v * w["scales"][e].double()[:, None]
    q = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=codes.device)
    q[:, 0::2], q[:, 1::2] = (codes % 16).double(), (codes // 16).double()
    scale = w["scales"][e].repeat_interleave(group, 1).double()
    if fmt == "mxfp4":
        sign, m = 1 - 2 * (q >= 8).double(), q % 8
        mag = torch.where(m < 2, m / 2, (1 + m % 2 / 2) * torch.exp2(torch.div(m, 2, rounding_mode="floor") - 1))
        return sign * mag * torch.exp2(scale - 127)
    if fmt == "int4":
        return (q - 16 * (q >= 8).double()) * scale
    return (q - w["zeros"][e].repeat_interleave(group, 1).double()) * scale


def _gated64(y):
    n = y.shape[-1] // 2
    return y[..., :n] * torch.sigmoid(y[..., :n]) * y[..., n:]


def exact(case, seed):
    c, m = case, _made(case, seed)
    if c["op"] == "route":
        if c["T"] > 4096:
            return None
        rows = m["logits"].double().cpu().tolist()
        bias = [0.0] * c["E"] if m["bias"] is None else m["bias"].double().cpu().tolist()
        per, found = c["E"] // c["groups"], {"ids": [], "weights": []}
        for row in rows:
            live = [e for e in range(c["E"]) if row[e] > -math.inf]
            most = max((row[e] for e in live), default=0.0)
            if c["sigmoid"]:
                score = {e: 1 / (1 + math.exp(-row[e])) for e in live}
            else:
                total = math.fsum(math.exp(row[e] - most) for e in live)
                score = {e: math.exp(row[e] - most) / total for e in live}
            value = {e: score[e] + bias[e] for e in live}
            best = {}
            for e in live:
                best.setdefault(e // per, []).append(value[e])
            kept = sorted(best, key=lambda b: (-sum(sorted(best[b])[-2:]), b))[: c["keep"]]
            by = {e: row[e] if m["bias"] is None else value[e] for e in live if c["groups"] == 1 or e // per in kept}
            ids = sorted(by, key=lambda e: (-by[e], e))[: c["topk"]]
            w = [score[e] for e in ids]
            total = math.fsum(w) if c["renorm"] else 1.0
            more = c["topk"] - len(ids)
            found["ids"].append(ids + [-1] * more)
            found["weights"].append([SCALE * v / total if total else 0.0 for v in w] + [0.0] * more)
        return {"ids": torch.tensor(found["ids"], dtype=torch.int32), "weights": torch.tensor(found["weights"], dtype=torch.float64)}
    x = m["x"].double()
    if c["op"] == "gemv":
        y = x @ _expert64(m["w"], 0, c["fmt"], c["group"]).T
        return _gated64(y) if c["gated"] else y
    out = torch.zeros_like(x)
    for e in m["ids"].unique().tolist():
        t, j = (m["ids"] == e).nonzero(as_tuple=True)
        act = _gated64(x[t] @ _expert64(m["gate_up"], e, c["fmt"], c["group"]).T)
        out.index_add_(0, t, m["weights"][t, j].double()[:, None] * (act @ _expert64(m["down"], e, c["fmt"], c["group"]).T))
    return out


# ---- what a case cannot do without ------------------------------------------------------------


def _weight_bytes(N, K, fmt, group):
    if fmt in ("int8", "fp8"):
        return N * K + 4 * N
    return N * K // 2 + N * K // group * {"mxfp4": 1, "int4": 2, "uint4": 2.5}[fmt]


def work(case):
    c = case
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * (2 if c["bf16"] else 4) + 8 * c["topk"]) + 4 * c["E"] * c["bias"], "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "gemv":
        out = c["N"] // (2 if c["gated"] else 1)
        return {"bytes": _weight_bytes(c["N"], c["K"], c["fmt"], c["group"]) + 2 * c["M"] * (c["K"] + out), "flops": 2 * c["M"] * c["N"] * c["K"]}
    H, I, T, k = c["H"], c["I"], c["T"], c["topk"]
    # experts that T tokens with k distinct experts each reach on average
    used = c["E"] * (1 - (1 - k / c["E"]) ** T)
    one = _weight_bytes(2 * I, H, c["fmt"], c["group"]) + _weight_bytes(H, I, c["fmt"], c["group"])
    return {"bytes": used * one + T * (4 * H + 8 * k), "flops": 6 * T * k * H * I}
