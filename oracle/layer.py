"""What stands around a decoder layer's products, for the oracle (test infrastructure): the RMS norm with the
residual's addition and quantized output, the append to a paged 8-bit cache of keys and values, and
attention over it.

Codes are integers decided by floating point, and the library takes those decisions in binary32 from
values that a stated sequence of roundings gives; the reference takes the same sequence (numpy's float32
operations are IEEE ones). Everything else is float64.
"""
from __future__ import annotations

import numpy as np

from .actquant import _mx_block_exponent, encode_e2m1, encode_e4m3
from .codecs import decode_bf16, decode_e4m3, decode_int8, round_to_bf16


def ref_rms_norm(x: np.ndarray, residual, weight, eps: float):
    """bf16 bits in. h = bf16(x + residual) (bits), and v = (h * r) * weight as float32, r = 1 / sqrt(mean h^2 + eps)."""
    if residual is not None:
        with np.errstate(invalid="ignore", over="ignore"):
            x = round_to_bf16(decode_bf16(x).astype(np.float32) + decode_bf16(residual).astype(np.float32))
    h = decode_bf16(x)
    with np.errstate(invalid="ignore"):
        r = (1.0 / np.sqrt((h * h).sum(1, keepdims=True) / h.shape[1] + float(np.float32(eps)))).astype(np.float32)
        v = h.astype(np.float32) * r
    if weight is not None:
        v = v * decode_bf16(weight).astype(np.float32)
    return x, v


def _scaled(v: np.ndarray, largest: float):
    """(v / s, s) with s = fp32(max |v| * fp32(1 / largest)) over the last axis, 1 where that is 0."""
    s = np.abs(v).max(-1).astype(np.float32) * (np.float32(1) / np.float32(largest))
    s = np.where(s == 0, np.float32(1), s).astype(np.float32)
    return (v / s[..., None]).astype(np.float32), s


def quantize_values(v: np.ndarray, fmt: str):
    """Codes and scales of float32 values [M, K]: "int8" and "fp8" by row, "block" by 128 columns, "mxfp8" and
    "mxfp4" by 32 with a power of two."""
    M, K = v.shape
    if fmt == "int8":
        q, s = _scaled(v, 127.0)
        return np.clip(np.rint(q), -127, 127).astype(np.int8), s
    if fmt == "fp8":
        q, s = _scaled(v, 448.0)
        return encode_e4m3(np.clip(q, np.float32(-448), np.float32(448))), s
    if fmt == "block":
        q, s = _scaled(v.reshape(M, K // 128, 128), 448.0)
        return encode_e4m3(np.clip(q, np.float32(-448), np.float32(448))).reshape(M, K), s
    blocks = v.astype(np.float64).reshape(M, K // 32, 32)
    if fmt == "mxfp8":
        e = _mx_block_exponent(blocks, 8)
        return encode_e4m3(np.clip(blocks * np.ldexp(1.0, -e)[:, :, None], -448, 448)).reshape(M, K), (e + 127).astype(np.uint8)
    e = _mx_block_exponent(blocks, 2)
    c = encode_e2m1(blocks * np.ldexp(1.0, -e)[:, :, None]).reshape(M, K)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), (e + 127).astype(np.uint8)


# ---- the cache ----------------------------------------------------------------------------------
UNIT = {"fp8": np.float32(1) / np.float32(448), "int8": np.float32(1) / np.float32(127)}


def _codes(q: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "int8":
        return np.clip(np.rint(q), -127, 127).astype(np.int8).view(np.uint8)
    return encode_e4m3(np.clip(q, np.float32(-448), np.float32(448)))


def _values(codes: np.ndarray, fmt: str) -> np.ndarray:
    return decode_int8(codes.view(np.int8)).astype(np.float64) if fmt == "int8" else decode_e4m3(codes)


def _sequences(cu, lens, T: int, most: int, capacity: int):
    """(sequence, first row, new tokens, length) of those that are not left out."""
    for b, length in enumerate(lens):
        first, end = int(cu[b]), int(cu[b + 1])
        if first >= 0 and first < end <= T and end - first <= most and 0 <= length <= capacity:
            yield b, first, end - first, int(length)


def ref_kv_append(fmt: str, x: np.ndarray, is_value: bool, cu, lens, table, pages: np.ndarray, scales: np.ndarray, max_new=None):
    """One of the two caches after an append. x: bf16 bits [T, H, D]; pages: code bytes [n, H, P, D], for values
    [n, H, D, P]; scales float32 [n, H]. Token by token within a page; returns new arrays."""
    pages, scales = pages.copy(), scales.copy()
    T, H, D = x.shape
    P = pages.shape[3] if is_value else pages.shape[2]
    for b, first, n, length in _sequences(cu, lens, T, T if max_new is None else max_new, table.shape[1] * P):
        start = max(length - n, 0)
        for p in range(start // P, -(-length // P)):
            page, lo, hi = int(table[b, p]), max(start, p * P), min(length, (p + 1) * P)
            if not 0 <= page < len(pages):
                continue
            rows = first + np.arange(lo, hi) - (length - n)
            for h in range(H):
                bits = x[rows, h]
                nan = (bits & 0x7FFF) > 0x7F80
                bits = np.where((bits & 0x7FFF) == 0x7F80, bits - 1, bits)       # infinities
                v = np.where(nan, 0.0, decode_bf16(np.where(nan, 0, bits).astype(np.uint16))).astype(np.float32)
                need = np.abs(v).max() * UNIT[fmt]
                old = pages[page, h].T if is_value else pages[page, h]           # [P, D], a view
                s = need
                if lo > p * P and scales[page, h] != 0:
                    s, e = scales[page, h], 0
                    while need > np.float32(np.ldexp(s, e)):
                        e += 1
                    if e:
                        c = old[:lo - p * P]
                        keep = (c & 0x7F) == 0x7F if fmt == "fp8" else np.zeros(c.shape, bool)
                        moved = _codes(np.where(keep, 0.0, _values(np.where(keep, 0, c).astype(np.uint8), fmt)) * 2.0 ** -e, fmt)
                        # the sign of a value that rounds to zero stays
                        old[:lo - p * P] = np.where(keep, c, moved)
                    s = np.float32(np.ldexp(s, e))
                scales[page, h] = s
                c = np.zeros(v.shape, np.uint8) if s == 0 else _codes((v / s).astype(np.float32), fmt)
                old[lo - p * P:hi - p * P] = np.where(nan, 0x7F if fmt == "fp8" and not is_value else 0, c)
    return pages, scales


def ref_attention(fmt: str, q: np.ndarray, cu, lens, table, k_pages, v_pages, k_scales, v_scales, sm_scale: float, window: int, out: np.ndarray,
                  max_q=None):
    """Attention row by row in float64. q: bf16 bits [T, Hq, D]; out: float64 [T, Hq, D], rows that are left out keep what
    they hold. Returns (out, size, spread, grain, reach) with, per output value, size = sum p |v| / sum p and spread = sqrt(sum
    (p v)^2) / sum p (which bound the effect of rounding each weight p * scale relative to itself), grain = max (p * scale)
    * sum |code| / sum p (relative to the row's largest), and per row reach = max over the seen j of sm_scale * sum |q k|
    (which bounds that of rounding in the scores)."""
    out = out.copy()
    T, Hq, D = q.shape
    n, H, P, _ = k_pages.shape
    size, spread, grain, reach = np.zeros(out.shape), np.zeros(out.shape), np.zeros(out.shape), np.zeros((T, Hq))
    qv = decode_bf16(q)
    for b, first, count, length in _sequences(cu, lens, T, T if max_q is None else max_q, table.shape[1] * P):
        j = np.arange(length)
        page = table[b, j // P] if length else np.zeros(0, int)
        there = (page >= 0) & (page < n)
        at = np.where(there, page, 0)
        for h in range(H):
            # codes of slots that hold nothing may be anything: only what a row sees enters
            with np.errstate(invalid="ignore"):
                k = _values(k_pages[at, h, j % P], fmt) * k_scales[at, h].astype(np.float64)[:, None]
                code, scale = _values(v_pages[at, h, :, j % P], fmt), v_scales[at, h].astype(np.float64)
                v = code * scale[:, None]
            for i in range(count):
                pos = length - count + i
                seen = there & (j <= pos) & ((j > pos - window) if window else True)
                for g in range(Hq // H):
                    r, c = first + i, h * (Hq // H) + g
                    if not seen.any():
                        out[r, c] = 0.0
                        continue
                    s = sm_scale * (k[seen] @ qv[r, c])
                    p = np.exp(s - s.max())
                    out[r, c] = p @ v[seen] / p.sum()
                    size[r, c] = p @ np.abs(v[seen]) / p.sum()
                    spread[r, c] = np.sqrt((p * p) @ (v[seen] ** 2)) / p.sum()
                    grain[r, c] = (p * scale[seen]).max() * np.abs(code[seen]).sum(0) / p.sum()
                    reach[r, c] = abs(sm_scale) * (np.abs(k[seen]) @ np.abs(qv[r, c])).max()
    return out, size, spread, grain, reach
