"""Inputs and bounds shared by the tests of the norm, the cache and the attention over it: caches in use with their tables,
and the error bounds of the attention derived from its arithmetic."""
from __future__ import annotations

import numpy as np

import oracle
import quantized_gemm_prepacked_amd as hq
import synth

KV = {"fp8": hq.HQ_KV_FP8_E4M3, "int8": hq.HQ_KV_INT8}
NORM = {"bf16": hq.HQ_ACT_BF16, "int8": hq.HQ_ACT_INT8_PER_TOKEN, "fp8": hq.HQ_ACT_FP8E4M3_PER_TOKEN,
        "block": hq.HQ_ACT_FP8E4M3_BLOCK128, "mxfp8": hq.HQ_ACT_MXFP8, "mxfp4": hq.HQ_ACT_MXFP4}


def kv_case(g: np.random.Generator, fmt: str, H: int, D: int, P: int, new: list, lens: list, spare: int = 3, peaky: float = 1.0, behind: int = 0):
    """A cache whose first lens - new tokens of each sequence are stored, in pages of no order, and all tokens' codes
    drawn at random; every byte that belongs to no stored token is 0xFF (a NaN in e4m3, -1 in INT8), every scale of no
    page in use NaN. `behind`: rows of the new tokens' tensors behind the last sequence."""
    held = [-(-n // P) for n in lens]
    width = max(held + [1]) + 1
    pages = sum(held) + spare
    order = g.permutation(pages)
    table = np.full((len(lens), width), -1, np.int32)
    k_pages = np.full((pages, H, P, D), 0xFF, np.uint8)
    v_pages = np.full((pages, H, D, P), 0xFF, np.uint8)
    k_scales = np.full((pages, H), np.nan, np.float32)
    v_scales = np.full((pages, H), np.nan, np.float32)
    at = 0

    def codes(shape):
        if fmt == "int8":
            return g.integers(-127, 128, shape).astype(np.int8).view(np.uint8)
        v = g.normal(0, 60, shape)
        return oracle.encode_e4m3(v)
    for b, n in enumerate(lens):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
        for p in range(held[b]):
            page, live = table[b, p], min(P, n - p * P)
            k_pages[page, :, :live] = codes((H, live, D))
            v_pages[page, :, :, :live] = codes((H, D, live))
            unit = 1 / 60
            k_scales[page] = (peaky * unit * g.uniform(0.5, 1.5, H)).astype(np.float32)
            v_scales[page] = (unit * g.uniform(0.5, 1.5, H)).astype(np.float32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return {"desc": hq.make_kv_desc(KV[fmt], H, D, P, pages), "fmt": fmt, "H": H, "D": D, "P": P, "B": len(lens), "T": int(cu[-1]) + behind,
            "max_new": max(new + [1]), "cu": cu, "lens": np.array(lens, np.int32), "table": table, "k_pages": k_pages, "v_pages": v_pages,
            "k_scales": k_scales, "v_scales": v_scales}


def attention_bounds(ref, size, spread, grain, reach, D: int, tokens: int):
    """(elementwise, squared per element) bounds of a result's error.
    Score: a dot product of D terms in fp32, each addition off by 2^-23 of the terms' size (a matrix instruction may
    truncate), and its two factors, the subtraction of the maximum and the exponential, together at most 8 steps more:
    each p off by 2 * 2^-23 (D + 8) reach relative (the factor 2 for the exponential's curvature and log2 e), plus 2^-21 for
    the exponential itself. p * scale as an fp16 relative to the row's largest: off by 2^-11 of itself or 2^-25 of that. Sums over the tokens: at most tokens / 32 + 40 additions one after
    another in a lane and 64 joins, 2^-23 each, of sum p |v| and sum p. The result rounded to bf16: 2^-8 of it, 2^-134 where
    it is subnormal.
    Squared: the rounding errors of the p's are independent, uniform at most: variance (2^-11)^2 / 3 of each (p v)^2;
    the result's (2^-8)^2 / 3 of its square, and (2^-134)^2 / 3 where it is subnormal (steps of 2^-133, so off by 2^-134 at
    most, whatever its size); the fp32 terms and the grain in full."""
    p = 2.0 ** -22 * (D + 8) * reach[..., None] + 2.0 ** -21
    chain = 2.0 ** -23 * (tokens / 32 + 104)
    fp32 = (p + chain) * (size + np.abs(ref))
    fp32 = fp32 + 2.0 ** -25 * grain
    hard = fp32 * 1.01 + 2.0 ** -11 * size * (1 + 2 * p)
    hard = hard + 2.0 ** -8 * (np.abs(ref) + hard) + 2.0 ** -134
    return hard, 2.0 ** -22 / 3 * spread ** 2 + 2.0 ** -16 / 3 * ref ** 2 + 2.0 ** -268 / 3 + fp32 ** 2


def check_attention(got, ref, size, spread, grain, reach, D, tokens, what, say=print):
    """Every element within the worst case; and the whole within twice the expected size of the errors (a lost or doubled
    token of n alike moves the result by 1 / sqrt(n) of its size)."""
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    hard, var = attention_bounds(ref, size, spread, grain, reach, D, tokens)
    err = np.abs(got - ref)
    worst = float((err / hard).max()) if err.size else 0.0
    rms = float(np.sqrt((err ** 2).sum() / var.sum())) if var.sum() > 0 else float(err.max() if err.size else 0.0)
    say(f"  {what}: worst {worst:.3f} of its bound, {rms:.3f} of the expected size")
    assert worst <= 1.0, what
    assert rms <= 2.0 or err.size < 256, what
    return worst, rms


def normal_rows(g, T, heads, D, std=1.0):
    return synth.normal_bf16(g, (T, heads, D), std)
