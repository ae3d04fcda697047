"""Oracle of the decode-step operators: the MoE router, matrix-vector products with packed weights and
the MoE layer for a few tokens -- plain fp64, row by row and expert by expert.

The announcement does not describe these steps; each is the operator's own definition (include/hq.h).
Weights come as dequantized fp64 arrays (``dequant_int4_groups`` here for INT4 groups of 32, 64 or 128;
the format functions of this package for the others)."""
from __future__ import annotations

import math

import numpy as np

from .codecs import decode_bf16, decode_int4_sym, decode_uint4, unpack_nibbles



def dequant_int4_groups(wq: np.ndarray, scales: np.ndarray, zeros, group: int) -> np.ndarray:
    """INT4 codes [N, K/2] (low nibble = even k), bf16 scale bits [N, K/group], zeros (or None: signed
    codes) -> fp64 [N, K]."""
    codes = unpack_nibbles(wq)
    q = (decode_int4_sym(codes) if zeros is None else decode_uint4(codes)).astype(np.float64)
    if zeros is not None:
        q = q - np.repeat(zeros.astype(np.float64), group, axis=-1)
    return q * np.repeat(decode_bf16(scales), group, axis=-1)


def ref_route(logits: np.ndarray, bias, score: str, topk: int, n_group: int = 1, topk_group: int = 1, group_top: int = 2,
              renormalize: bool = True, scale: float = 1.0):
    """logits [T, E] (taken in fp64) -> (ids int32 [T, topk], weights fp64 [T, topk])."""
    T, E = logits.shape
    per = E // n_group
    ids = np.full((T, topk), -1, np.int32)
    weights = np.zeros((T, topk))
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    for t in range(T):
        l = logits[t].astype(np.float64)
        on = [e for e in range(E) if l[e] > -math.inf and b[e] > -math.inf]       # False for NaN
        # switched off by the logit: not in the softmax's sum; by the bias alone: in it, never chosen
        live = [e for e in range(E) if l[e] > -math.inf]
        top = max((l[e] for e in live), default=0.0)
        if score == "sigmoid":
            s = {e: 1.0 / (1.0 + math.exp(-l[e])) if l[e] > -700 else math.exp(l[e]) for e in live}
        else:
            ex = {e: 1.0 if l[e] == top else math.exp(l[e] - top) for e in live}
            total = math.fsum(ex.values())
            s = {e: ex[e] / total for e in live}
        v = {e: s[e] + b[e] for e in on}
        groups = {}
        for e in on:
            groups.setdefault(e // per, []).append(v[e])
        value = {g: sum(sorted(vs, reverse=True)[:group_top]) for g, vs in groups.items()}
        kept = set(sorted(value, key=lambda g: (-value[g], g))[:topk_group])
        pick = sorted((e for e in on if e // per in kept), key=lambda e: (-(l[e] if bias is None else v[e]), e))[:topk]
        w = [s[e] for e in pick]
        total = math.fsum(w) if renormalize else 1.0
        for j, e in enumerate(pick):
            ids[t, j] = e
            weights[t, j] = scale * w[j] / total if total > 0 else 0.0
    return ids, weights


def ref_gemv(x_bits: np.ndarray, w: np.ndarray, gated: bool) -> np.ndarray:
    """bf16 bits [M, K] by fp64 [N, K] -> unrounded fp64 [M, N] (gated: silu(first half) * second half)."""
    y = decode_bf16(x_bits) @ w.T
    if not gated:
        return y
    n = y.shape[1] // 2
    return _silu(y[:, :n]) * y[:, n:]


def _silu(g: np.ndarray) -> np.ndarray:
    e = np.exp(-np.abs(g))
    return g * np.where(g >= 0, 1.0, e) / (1.0 + e)


def ref_moe_decode(x_bits: np.ndarray, ids: np.ndarray, weights, gate_up, down) -> np.ndarray:
    """x bf16 bits [T, H], ids [T, topk], weights [T, topk] or None, gate_up(e) / down(e): fp64 weights
    of expert e ([2I, H] / [H, I]), E experts = len of the id range the caller allows (ids outside are
    given as -1) -> unrounded fp64 [T, H]."""
    T, topk = ids.shape
    x = decode_bf16(x_bits)
    out = np.zeros(x.shape)
    for e in sorted({int(i) for i in ids.ravel() if i >= 0}):
        rows = [t for t in range(T) if e in ids[t]]
        gu = x[rows] @ gate_up(e).T
        n = gu.shape[1] // 2
        y = (_silu(gu[:, :n]) * gu[:, n:]) @ down(e).T
        for i, t in enumerate(rows):
            for j in range(topk):
                if ids[t, j] == e:
                    out[t] += (1.0 if weights is None else float(weights[t, j])) * y[i]
    return out


__all__ = ["dequant_int4_groups", "ref_route", "ref_gemv", "ref_moe_decode"]
