"""Inputs and bounds shared by the decode-step tests: random packed weights of every format with their
fp64 values, and the error bound of a matrix-vector product derived from its arithmetic."""
from __future__ import annotations

import numpy as np

import oracle
import quantized_gemm_prepacked_amd as hq
import synth

#: name -> (descriptor, group, zero-points)
FORMATS = {
    "int4_g32": (hq.DESC_W4A16_SYM_G32, 32, False),
    "uint4_g32": (hq.DESC_W4A16_ASYM_G32, 32, True),
    "int4_g64": (hq.DESC_W4A16_SYM_G64, 64, False),
    "uint4_g64": (hq.DESC_W4A16_ASYM_G64, 64, True),
    "int4_g128": (hq.DESC_W4A16_SYM, 128, False),
    "uint4_g128": (hq.DESC_W4A16_ASYM, 128, True),
    "mxfp4": (hq.DESC_W4A16_MXFP4, 32, False),
    "int8": (hq.DESC_W8A16_INT8, 0, False),
    "fp8": (hq.DESC_W8A16_FP8, 0, False),
}


def random_weights(g: np.random.Generator, fmt: str, N: int, K: int) -> dict:
    """Every code equally likely; scales spread over a factor of about three, zero and negative ones
    among the bf16 scales."""
    _, group, asym = FORMATS[fmt]
    if group and fmt != "mxfp4":
        s = g.uniform(0.02, 0.06, (N, K // group))
        s[g.random(s.shape) < 0.02] = 0.0
        s *= np.where(g.random(s.shape) < 0.1, -1, 1)
        return {"wq": g.integers(0, 256, (N, K // 2), dtype=np.uint8), "scales": synth.bf16_bits(s.astype(np.float32)),
                "zeros": g.integers(0, 16, (N, K // group), dtype=np.uint8) if asym else None}
    if fmt == "mxfp4":
        return {"wq": g.integers(0, 256, (N, K // 2), dtype=np.uint8),
                "scales": g.integers(118, 126, (N, K // 32), dtype=np.uint8), "zeros": None}
    s = g.uniform(0.001, 0.003, N).astype(np.float32)
    if fmt == "int8":
        return {"wq": g.integers(-127, 128, (N, K), dtype=np.int64).astype(np.int8), "scales": s, "zeros": None}
    c = g.integers(0, 256, (N, K), dtype=np.uint8)
    c[(c & 0x7F) == 0x7F] ^= 1      # 0x7f and 0xff are NaN
    return {"wq": c, "scales": s, "zeros": None}


def dequant(w: dict, fmt: str) -> np.ndarray:
    _, group, _ = FORMATS[fmt]
    if fmt == "mxfp4":
        return oracle.dequant_mxfp4(w["wq"], w["scales"])
    if fmt == "int8":
        return oracle.decode_int8(w["wq"]).astype(np.float64) * w["scales"].astype(np.float64)[:, None]
    if fmt == "fp8":
        return oracle.decode_e4m3(w["wq"]) * w["scales"].astype(np.float64)[:, None]
    return oracle.dequant_int4_groups(w["wq"], w["scales"], w["zeros"], group)


def magnitude(w: dict, fmt: str) -> np.ndarray:
    """Per weight, the size of what the kernel accumulates for it: INT4 products are formed as
    x (128 + q) - (128 + z) x, both below 144 |x| before the scale; every other weight is exact."""
    _, group, _ = FORMATS[fmt]
    if fmt.startswith(("int4", "uint4")):
        return 288.0 * np.repeat(np.abs(oracle.decode_bf16(w["scales"])), group, axis=-1)
    return np.abs(dequant(w, fmt))


def product_bound(x: np.ndarray, w: dict, fmt: str) -> np.ndarray:
    """fp32 error of x . w^T (x: bf16 bits or fp64 values) before its rounding to bf16. Every partial sum is at most A = sum_k |x_k|
    |w_k|'s accumulated size; a product passes through at most 128 additions inside its scale group's
    matrix instructions, K/128 over the units, 16 waves, and 8 more for scaling, channel scales and
    router weights, each off by 2^-24 relative (2^-23 here: a matrix instruction may truncate)."""
    K = x.shape[1]
    a = np.abs(oracle.decode_bf16(x) if x.dtype == np.uint16 else x) @ magnitude(w, fmt).T
    return 2.0 ** -23 * (128 + K // 128 + 16 + 8) * a


def group_product_bound(x: np.ndarray, w: dict, fmt: str) -> np.ndarray:
    """product_bound for long K, where INT4's offset form must not be charged to the whole sum. A group's two
    offset sums, sum x (128 + q) and (128 + z) sum x, stay apart from the others: each of their terms (together
    below 288 |x| before the scale) passes through at most G additions, and 8 more for the halves of a row, the
    subtraction and the scale. What is added up over the K / G groups, 16 waves and 8 more steps is the groups'
    values themselves, at most sum |x w|. Both at 2^-23 a step, as there; errors of errors: 2^-6 of it."""
    _, group, _ = FORMATS[fmt]
    if not fmt.startswith(("int4", "uint4")):
        return product_bound(x, w, fmt)
    ax = np.abs(oracle.decode_bf16(x) if x.dtype == np.uint16 else x)
    offsets = (group + 8) * (ax @ magnitude(w, fmt).T)
    chain = (x.shape[1] // group + 24) * (ax @ np.abs(dequant(w, fmt)).T)
    return 2.0 ** -23 * (1 + 2.0 ** -6) * (offsets + chain)


def prepack_host(desc, w: dict, N: int, K: int) -> np.ndarray:
    stack = w if isinstance(w, list) else [w]
    out = np.zeros(hq.hq_decode_prepacked_bytes(desc, len(stack), N, K), np.uint8)
    zeros = None if stack[0]["zeros"] is None else np.stack([e["zeros"] for e in stack])
    return hq.hq_decode_prepack_weights(desc, len(stack), N, K, np.stack([e["wq"] for e in stack]),
                                        np.stack([e["scales"] for e in stack]), zeros, out)


def route_case(g: np.random.Generator, T: int, E: int, bf16: bool, masked: float = 0.0, special: bool = False):
    """Logits as fp32 values (bf16-representable if bf16); switched-off ones, and with special rows of
    nothing but -inf or NaN, infinities, equal logits and large ones."""
    l = g.normal(0, 2, (T, E)).astype(np.float32)
    l[g.random((T, E)) < masked] = -np.inf
    if special:
        kinds = [lambda r: r.fill(-np.inf), lambda r: r.fill(np.nan), lambda r: r.fill(0.25),
                 lambda r: r.__setitem__(slice(None, None, 3), np.nan), lambda r: r.__setitem__(slice(0, 2), np.inf),
                 lambda r: r.__imul__(60.0), lambda r: r.__setitem__(slice(1, None), -np.inf)]
        with np.errstate(invalid="ignore"):
            for t in range(min(T, len(kinds))):
                kinds[t](l[t])
    if bf16:
        l = synth.bf16_bits_to_f32(synth.bf16_bits(l))
    return l
