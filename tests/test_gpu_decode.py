"""GPU parity of the decode-step calls (router, matrix-vector products, MoE layer for a few tokens)
against the fp64 oracle, and of a whole decode step built from them."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_prepacked_amd as hq
import synth

from decode_harness import FORMATS, dequant, group_product_bound, magnitude, prepack_host, product_bound, random_weights, route_case
from gpu_harness import BF16_NAN_BITS, DEV, bf16_to_f64, check_float, say, to_dev

pytestmark = pytest.mark.gpu

PAD = 256   # canary elements behind every output


def _out(shape):
    n = int(np.prod(shape))
    flat = torch.full((n + PAD,), BF16_NAN_BITS, dtype=torch.int16, device=DEV)
    return flat, flat[:n].view(shape)


def _bits(t):
    return t.cpu().numpy().view(np.uint16)


def _untouched(flat, n):
    assert bool((flat[n:] == BF16_NAN_BITS).all()), "written behind the output"


def _check(got_bits, ref64, fp32_bound, what):
    """Each value within half a bf16 step (2^-8 relative) of the exact one moved by the fp32 bound."""
    got = bf16_to_f64(got_bits)
    err, bound = np.abs(got - ref64), fp32_bound + 2.0 ** -8 * (np.abs(ref64) + fp32_bound) + 2.0 ** -134
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    worst = float((err / bound).max())
    say(f"  {what}: worst error {worst:.3f} of its bound")
    assert worst <= 1.0, what


# ---- router -----------------------------------------------------------------------------------
def _route(l, bias, score, topk, bf16, **k):
    T, E = l.shape
    dev = torch.from_numpy(l).to(DEV).to(torch.bfloat16 if bf16 else torch.float32)
    ids = torch.full((T * topk + PAD,), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T * topk + PAD,), 7.5, dtype=torch.float32, device=DEV)
    hq.hq_moe_route(hq.HQ_SCORE_SIGMOID if score == "sigmoid" else hq.HQ_SCORE_SOFTMAX, T, E, topk, dev,
                    hq.HQ_LOGITS_BF16 if bf16 else hq.HQ_LOGITS_FP32, None if bias is None else to_dev(bias),
                    k.get("n_group", 1), k.get("topk_group", 1), k.get("group_top", 2), k.get("renormalize", True),
                    k.get("scale", 1.0), ids, w)
    torch.cuda.synchronize()
    assert bool((ids[T * topk:] == 77).all()) and bool((w[T * topk:] == 7.5).all()), "written behind the output"
    return ids[:T * topk].view(T, topk).cpu().numpy(), w[:T * topk].view(T, topk).cpu().numpy()


def _check_route(l, bias, score, topk, bf16, **k):
    ids, w = _route(l, bias, score, topk, bf16, **k)
    want_ids, want = oracle.ref_route(l.astype(np.float64), bias, score, topk, **k)
    assert np.array_equal(ids, want_ids), f"first wrong row {np.argwhere((ids != want_ids).any(1))[0]}"
    # 64-bit scores rounded once to fp32: half a step, 2^-24 relative (2^-150 among the subnormals); the
    # 64-bit exp, sum over at most 512 and division move that by less than 2^-40
    assert (np.abs(w - want) <= 2.0 ** -24 * (1 + 2.0 ** -10) * np.abs(want) + 2.0 ** -150).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,topk,bf16", [(1, 1, 1, False), (1, 256, 8, False), (3, 60, 4, True), (5, 64, 64, False),
                                           (9, 65, 6, True), (130, 128, 1, False), (7, 257, 8, False), (33, 512, 16, True),
                                           (1, 512, 64, False)])
def test_route(score, T, E, topk, bf16):
    g = np.random.default_rng(100 + T + E)
    for masked in (0.0, 0.3):
        l = route_case(g, T, E, bf16, masked)
        say(f"[route] {score} T={T} E={E} topk={topk} bf16={bf16} masked={masked}")
        _check_route(l, None, score, topk, bf16, renormalize=masked > 0, scale=1.5)
        _check_route(l, g.normal(0, 0.05, E).astype(np.float32), score, topk, bf16)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,topk", [(256, 8, 4, 8), (64, 64, 5, 5), (96, 2, 1, 48), (512, 64, 64, 8),
                                                       (60, 4, 3, 6), (6, 3, 2, 4), (320, 5, 2, 64)])
def test_route_groups(score, E, n_group, topk_group, topk):
    g = np.random.default_rng(200 + E)
    for bias in (None, g.normal(0, 0.1, E).astype(np.float32)):
        for group_top, masked in ((2, 0.0), (1, 0.2), (2, 0.6)):
            l = route_case(g, 21, E, False, masked)
            say(f"[route groups] {score} E={E} groups={n_group}/{topk_group} top={group_top} masked={masked} bias={bias is not None}")
            _check_route(l, bias, score, topk, False, n_group=n_group, topk_group=topk_group, group_top=group_top, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n_group,topk_group", [(1, 1), (4, 2)])
def test_route_special_rows(score, bf16, n_group, topk_group):
    """Rows that leave nothing, NaN and infinite logits, ties, far-apart logits; switched-off biases."""
    g = np.random.default_rng(300)
    l = route_case(g, 12, 40, bf16, 0.1, special=True)
    bias = g.normal(0, 0.1, 40).astype(np.float32)
    bias[[3, 17]] = -np.inf, np.nan
    for b in (None, bias):
        for renorm in (False, True):
            _check_route(l, b, score, 7, bf16, n_group=n_group, topk_group=topk_group, renormalize=renorm)


def test_route_ties_take_the_lowest_id():
    l = np.zeros((2, 300), np.float32)
    l[1, [5, 70, 299]] = 1.0
    ids, _ = _route(l, None, "softmax", 4, False)
    assert ids.tolist() == [[0, 1, 2, 3], [5, 70, 299, 0]]


@pytest.mark.parametrize("bias,n_group,topk_group", [(False, 1, 1), (True, 1, 1), (False, 4, 2)])
def test_route_sigmoid_far_below_zero(bias, n_group, topk_group):
    """Rows of nothing but logits whose exp(-l) binary64 does not hold, though it holds their sigmoids: the
    weights are the scores' shares all the same. (At -720 a subnormal score has 35 bits left, so the check's
    2^-24 of a weight stands.)"""
    g = np.random.default_rng(450)
    l = g.uniform(-720, -650, (6, 40)).astype(np.float32)
    l[:3] = g.uniform(-720, -711, (3, 40))
    l[5, 1:] = -np.inf
    l[5, 0] = -715.0
    _check_route(l, np.zeros(40, np.float32) if bias else None, "sigmoid", 5, False, n_group=n_group, topk_group=topk_group)


def test_route_many_rows():
    g = np.random.default_rng(400)
    l = route_case(g, 5000, 128, True)
    ids, w = _route(l, None, "softmax", 8, True)
    order = np.argsort(-l, axis=1, kind="stable")[:, :8]
    assert np.array_equal(ids, order)
    e = np.exp(np.take_along_axis(l, order, 1).astype(np.float64))
    assert np.allclose(w, e / e.sum(1, keepdims=True), rtol=1e-6, atol=0)


# ---- matrix-vector products -------------------------------------------------------------------
def _gemv(desc, gated, x_bits, packed, N, K):
    M, outs = x_bits.shape[0], N // 2 if gated else N
    flat, y = _out((M, outs))
    hq.hq_gemv(desc, hq.HQ_GEMV_SILU_MUL if gated else hq.HQ_GEMV_LINEAR, M, N, K, to_dev(x_bits.view(np.int16)), packed, y)
    torch.cuda.synchronize()
    _untouched(flat, M * outs)
    return _bits(y)


def _gated_bound(x, w, fmt, N):
    """|d(silu(g) u)| <= 1.1 |u| dg + |silu(g)| du + 1.1 dg du (|silu'| < 1.1), and 8 fp32 roundings of
    the activation itself (exp and division included)."""
    b = product_bound(x, w, fmt)
    y = oracle.ref_gemv(x, dequant(w, fmt), False)
    g, u, dg, du = y[:, :N // 2], y[:, N // 2:], b[:, :N // 2], b[:, N // 2:]
    s = g / (1 + np.exp(-np.clip(g, -700, 700)))
    return 1.1 * np.abs(u) * dg + np.abs(s) * du + 1.1 * dg * du + 2.0 ** -21 * np.abs(s * u)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (1, 272, 1152), (2, 48, 256), (3, 4112, 384), (4, 256, 4096), (5, 32, 2944),
                                   (8, 528, 512), (13, 96, 640), (16, 256, 2048), (17, 48, 256), (50, 80, 384)])
def test_gemv(fmt, M, N, K):
    g = np.random.default_rng(1000 + M + N + K)
    w = random_weights(g, fmt, N, K)
    x = synth.normal_bf16(g, (M, K))
    packed = to_dev(prepack_host(FORMATS[fmt][0], w, N, K))
    say(f"[gemv] {fmt} M={M} N={N} K={K}")
    ref = oracle.ref_gemv(x, dequant(w, fmt), False)
    got = _gemv(FORMATS[fmt][0], False, x, packed, N, K)
    _check(got, ref, product_bound(x, w, fmt), "linear")
    check_float(got, ref, "linear", rounding_floor=True)
    if N % 32 == 0:
        ref = oracle.ref_gemv(x, dequant(w, fmt), True)
        got = _gemv(FORMATS[fmt][0], True, x, packed, N, K)
        _check(got, ref, _gated_bound(x, w, fmt, N), "gated")
        check_float(got, ref, "gated", rounding_floor=True)


@pytest.mark.parametrize("M,N,K,gated", [(1, 8208, 128, False), (4, 8208, 256, False), (16, 8208, 128, False),   # three tiles a workgroup
                                         (16, 12304, 128, False), (9, 8224, 128, True),                      # four
                                         (1, 64, 8192, True), (1, 4096, 2176, False), (1, 32, 16384, False)])
@pytest.mark.parametrize("fmt", ["uint4_g128", "int4_g64", "uint4_g32", "mxfp4", "int8"])
def test_gemv_workgroup_shapes(fmt, M, N, K, gated):
    """Sizes that take the other tile counts, waves and ring depths."""
    g = np.random.default_rng(1050 + N)
    w = random_weights(g, fmt, N, K)
    x = synth.normal_bf16(g, (M, K))
    say(f"[gemv shapes] {fmt} M={M} N={N} K={K} gated={gated}")
    got = _gemv(FORMATS[fmt][0], gated, x, to_dev(prepack_host(FORMATS[fmt][0], w, N, K)), N, K)
    ref = oracle.ref_gemv(x, dequant(w, fmt), gated)
    _check(got, ref, _gated_bound(x, w, fmt, N) if gated else product_bound(x, w, fmt), "shapes")
    check_float(got, ref, "shapes", rounding_floor=True)


def test_gemv_large():
    """The sizes a model has: a wide projection, sampled against the oracle."""
    g = np.random.default_rng(1100)
    for fmt, M, N, K in (("uint4_g64", 1, 14336, 4096), ("int4_g32", 3, 4096, 14336), ("uint4_g128", 13, 8208, 8192)):
        w = random_weights(g, fmt, N, K)
        x = synth.normal_bf16(g, (M, K))
        say(f"[gemv large] {fmt} M={M} N={N} K={K}")
        got = _gemv(FORMATS[fmt][0], False, x, to_dev(prepack_host(FORMATS[fmt][0], w, N, K)), N, K)
        cols = np.unique(np.concatenate([g.integers(0, N, 200), [0, 15, 16, N - 1]]))
        part = {k: None if v is None else v[cols] for k, v in w.items()}
        _check(got[:, cols], oracle.ref_gemv(x, dequant(part, fmt), False), product_bound(x, part, fmt), "sampled")


@pytest.mark.parametrize("fmt,M,N,K", [("uint4_g64", 1, 14336, 4096), ("int4_g32", 3, 4096, 14336), ("uint4_g128", 13, 8208, 8192),
                                       ("uint4_g32", 16, 12304, 4096)])     # the last: four tiles a workgroup
def test_gemv_large_loses_nothing(fmt, M, N, K):
    """The sizes a model has, by checks that a lost scale group and a lost k break (the host test of the
    large products' checks plants both in the oracle)."""
    g = np.random.default_rng(1150 + M)
    w = random_weights(g, fmt, N, K)
    x = synth.normal_bf16(g, (M, K))
    say(f"[gemv large] {fmt} M={M} N={N} K={K}")
    got = _gemv(FORMATS[fmt][0], False, x, to_dev(prepack_host(FORMATS[fmt][0], w, N, K)), N, K)
    cols = np.unique(np.concatenate([g.integers(0, N, 200), [0, 15, 16, N - 1]]))
    part = {k: None if v is None else v[cols] for k, v in w.items()}
    ref = oracle.ref_gemv(x, dequant(part, fmt), False)
    _check(got[:, cols], ref, group_product_bound(x, part, fmt), "sampled")
    check_float(got[:, cols], ref, "sampled")


def test_gemv_equals_gemm_weights():
    """Weights packed once serve hq_gemm and hq_gemv."""
    g = np.random.default_rng(1200)
    w = random_weights(g, "uint4_g128", 256, 512)
    x = synth.normal_bf16(g, (4, 512))
    packed = to_dev(prepack_host(hq.DESC_W4A16_ASYM, w, 256, 512))
    from gpu_harness import gemm
    ref = oracle.ref_gemv(x, dequant(w, "uint4_g128"), False)
    check_float(gemm(hq.DESC_W4A16_ASYM, 4, 256, 512, to_dev(x.view(np.int16)), None, packed), ref, "hq_gemm")
    check_float(_gemv(hq.DESC_W4A16_ASYM, False, x, packed, 256, 512), ref, "hq_gemv")


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("M", [2, 4, 7, 16])
def test_gemv_rows_do_not_mix(fmt, M):
    """NaN and infinity in one row leave the others as they were, bit for bit."""
    g = np.random.default_rng(1300)
    N, K = 64, 640
    w = random_weights(g, fmt, N, K)
    x = synth.normal_bf16(g, (M, K))
    packed = to_dev(prepack_host(FORMATS[fmt][0], w, N, K))
    for gated in (False, True):
        clean = _gemv(FORMATS[fmt][0], gated, x, packed, N, K)
        bad = x.copy()
        bad[M - 1, :] = 0x7FC0
        bad[0, 7] = 0x7F80
        got = _gemv(FORMATS[fmt][0], gated, bad, packed, N, K)
        assert np.array_equal(got[1:M - 1], clean[1:M - 1])
        assert not np.isfinite(bf16_to_f64(got[M - 1])).any()


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("M", [2, 3, 4, 5, 16, 17])
def test_gemv_one_bad_row(fmt, M):
    """One bad row at a time, so that every other row is compared while clean: NaN in the last one, which a block
    of rows repeats in its unused places, and infinity in the first. M = 17: a second block, of one row."""
    g = np.random.default_rng(1350)
    N, K = 64, 640
    w = random_weights(g, fmt, N, K)
    x = synth.normal_bf16(g, (M, K))
    packed = to_dev(prepack_host(FORMATS[fmt][0], w, N, K))
    for gated in (False, True):
        clean = _gemv(FORMATS[fmt][0], gated, x, packed, N, K)
        assert np.isfinite(bf16_to_f64(clean)).all()
        for row, at, bits in ((M - 1, slice(None), 0x7FC0), (M - 1, 639, 0x7FC0), (0, 7, 0x7F80)):
            bad = x.copy()
            bad[row, at] = bits
            got = _gemv(FORMATS[fmt][0], gated, bad, packed, N, K)
            rest = np.arange(M) != row
            assert rest.any() and np.array_equal(got[rest], clean[rest]), (gated, row)
            assert not np.isfinite(bf16_to_f64(got[row])).all()


def test_gated_extremes():
    """Gates far out on both sides: silu keeps its tiny products and never divides infinities."""
    g = np.random.default_rng(1400)
    N, K = 64, 128
    w = random_weights(g, "int8", N, K)
    x = (synth.normal_bf16(g, (4, K)).astype(np.uint32) << 16).view(np.float32)
    x *= np.array([1e-20, 1.0, 50.0, 1e10], np.float32)[:, None]
    xb = synth.bf16_bits(x)
    got = _gemv(hq.DESC_W8A16_INT8, True, xb, to_dev(prepack_host(hq.DESC_W8A16_INT8, w, N, K)), N, K)
    ref = oracle.ref_gemv(xb, dequant(w, "int8"), True)
    # below fp32's range exp(-|g|) is a subnormal or zero: an absolute error of 2^-149 carried by |g u|
    y = oracle.ref_gemv(xb, dequant(w, "int8"), False)
    _check(got, ref, _gated_bound(xb, w, "int8", N) + 2.0 ** -148 * np.abs(y[:, :N // 2] * y[:, N // 2:]), "extremes")


# ---- MoE layer --------------------------------------------------------------------------------
class Layer:
    def __init__(self, seed, fmt, E, H, I):
        g = np.random.default_rng(seed)
        self.fmt, self.desc, self.E, self.H, self.I = fmt, FORMATS[fmt][0], E, H, I
        self.gu = [random_weights(g, fmt, 2 * I, H) for _ in range(E)]
        self.dn = [random_weights(g, fmt, H, I) for _ in range(E)]
        self.gu_dev = to_dev(prepack_host(self.desc, self.gu, 2 * I, H))
        self.dn_dev = to_dev(prepack_host(self.desc, self.dn, H, I))

    def run(self, x_bits, ids, weights, out=None, ws=None, stream=None, x_dev=None):
        T, topk = ids.shape
        x = to_dev(x_bits.view(np.int16)) if x_dev is None else x_dev
        flat = None
        if out is None:
            flat, out = _out((T, self.H))
        if ws is None:
            n = hq.hq_moe_decode_workspace_bytes(self.desc, T, topk, self.E, self.H, self.I)
            ws = torch.full((n + PAD,), 0x7F, dtype=torch.uint8, device=DEV)   # NaN patterns, and a canary
        n = ws.numel() - PAD
        hq.hq_moe_decode(self.desc, T, topk, self.E, self.H, self.I, x, to_dev(ids), None if weights is None else to_dev(weights),
                         self.gu_dev, self.dn_dev, out, ws, n, stream)
        torch.cuda.synchronize()
        assert bool((ws[n:] == 0x7F).all()), "written behind the workspace"
        if flat is not None:
            _untouched(flat, T * self.H)
        return _bits(out)

    def ref(self, x_bits, ids, weights):
        ok = np.where((ids >= 0) & (ids < self.E), ids, -1)
        return oracle.ref_moe_decode(x_bits, ok, weights, lambda e: dequant(self.gu[e], self.fmt), lambda e: dequant(self.dn[e], self.fmt))

    def bound(self, x_bits, ids, weights):
        """Before the output's rounding: the down product's fp32 bound on the exact activations, and what
        the activations' own errors move -- their fp32 bound, and 2^-16 of each (a high and a low bf16: the
        low one is at most 2^-8 of the value and off by half a step, 2^-8, of itself; below bf16's range the
        low half is off by 2^-134) -- summed over the experts with their weights."""
        T, topk = ids.shape
        total = np.zeros((T, self.H))
        for t in range(T):
            for j in range(topk):
                e = int(ids[t, j])
                if not 0 <= e < self.E:
                    continue
                wt = 1.0 if weights is None else abs(float(weights[t, j]))
                xr = x_bits[t:t + 1]
                a64 = oracle.ref_gemv(xr, dequant(self.gu[e], self.fmt), True)
                moved = _gated_bound(xr, self.gu[e], self.fmt, 2 * self.I) + 2.0 ** -16 * np.abs(a64) + 2.0 ** -134
                d = np.abs(dequant(self.dn[e], self.fmt))
                total[t] += wt * (product_bound(a64, self.dn[e], self.fmt)[0] + (moved @ d.T)[0])
        return total + 2.0 ** -22 * topk * np.abs(total)


def _ids(g, T, topk, E):
    return np.stack([g.permutation(E)[:topk] for _ in range(T)]).astype(np.int32)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("T,topk,E,H,I", [(1, 1, 1, 128, 128), (1, 8, 16, 256, 384), (2, 2, 3, 384, 128), (3, 6, 8, 1152, 256),
                                          (4, 4, 9, 256, 640), (5, 3, 4, 128, 256), (11, 2, 32, 256, 128), (16, 8, 8, 384, 256),
                                          # the down products' items split over several workgroups
                                          (1, 8, 16, 128, 1024), (4, 8, 20, 256, 512), (16, 4, 40, 128, 640), (16, 6, 6, 256, 896)])
def test_moe_decode(fmt, T, topk, E, H, I):
    g = np.random.default_rng(2000 + T + H + I)
    L = Layer(2100 + T, fmt, E, H, I)
    x = synth.normal_bf16(g, (T, H))
    ids = _ids(g, T, topk, E)
    w = g.random((T, topk)).astype(np.float32)
    say(f"[moe decode] {fmt} T={T} topk={topk} E={E} H={H} I={I}")
    got, ref = L.run(x, ids, w), L.ref(x, ids, w)
    _check(got, ref, L.bound(x, ids, w), "layer")
    check_float(got, ref, "layer", rounding_floor=True)


@pytest.mark.parametrize("T", [1, 2, 4, 9, 16])
def test_moe_decode_odd_routing(T):
    """Ids outside [0, E), tokens with none left, an expert twice (or more) in a token's row, all tokens
    on one expert, no weights."""
    g = np.random.default_rng(2200 + T)
    E, H, I, topk = 6, 256, 128, 5
    L = Layer(2201, "uint4_g64", E, H, I)
    x = synth.normal_bf16(g, (T, H))
    w = g.random((T, topk)).astype(np.float32)
    cases = {"outside": g.integers(-2, E + 2, (T, topk)), "none": np.full((T, topk), -1), "same": np.full((T, topk), 3),
             "twice": np.tile([2, 0, 2, 5, 2], (T, 1)), "extremes": np.full((T, topk), 2 ** 31 - 1)}
    cases["mixed"] = cases["outside"].copy()
    cases["mixed"][T - 1] = (-1, E, -2 ** 31, 2 ** 31 - 1, E + 7)
    for name, ids in cases.items():
        ids = ids.astype(np.int32)
        for wt in (w, None):
            say(f"[moe decode] T={T} {name} weights={wt is not None}")
            got, ref = L.run(x, ids, wt), L.ref(x, ids, wt)
            _check(got, ref, L.bound(x, ids, wt), name)
            if name in ("none", "extremes"):
                assert not got.any()


@pytest.mark.parametrize("fmt", ["int4_g32", "int4_g128", "mxfp4", "fp8"])
@pytest.mark.parametrize("T", [2, 4, 13])
def test_moe_decode_tokens_do_not_mix(fmt, T):
    g = np.random.default_rng(2300)
    L = Layer(2301, fmt, 4, 256, 256)
    x = synth.normal_bf16(g, (T, 256))
    ids = _ids(g, T, 2, 4)
    w = g.random((T, 2)).astype(np.float32)
    clean = L.run(x, ids, w)
    bad = x.copy()
    bad[0] = 0x7FC0
    got = L.run(bad, ids, w)
    assert np.array_equal(got[1:], clean[1:]) and not np.isfinite(bf16_to_f64(got[0])).any()
    w2 = w.copy()
    w2[T - 1] = np.nan
    got = L.run(x, ids, w2)
    assert np.array_equal(got[:-1], clean[:-1])


def test_moe_decode_is_repeatable_and_in_place():
    g = np.random.default_rng(2400)
    L = Layer(2401, "int4_g128", 12, 512, 1408)
    for T in (1, 4, 16):
        x = synth.normal_bf16(g, (T, 512))
        ids, w = _ids(g, T, 4, 12), g.random((T, 4)).astype(np.float32)
        first = L.run(x, ids, w)
        for _ in range(5):
            assert np.array_equal(L.run(x, ids, w), first)
        buf = to_dev(x.view(np.int16))
        assert np.array_equal(L.run(x, ids, w, out=buf, x_dev=buf), first)     # out is x


def test_moe_decode_large_sampled():
    """One token and a full batch at a large model's expert size; four experts held."""
    g = np.random.default_rng(2500)
    L = Layer(2501, "int4_g128", 4, 7168, 2048)
    for T, topk in ((1, 4), (16, 2)):
        x = synth.normal_bf16(g, (T, 7168))
        ids, w = _ids(g, T, topk, 4), g.random((T, topk)).astype(np.float32)
        say(f"[moe decode large] T={T}")
        check_float(L.run(x, ids, w), L.ref(x, ids, w), f"T={T}")


@pytest.mark.parametrize("fmt", ["uint4_g64", "mxfp4", "fp8"])
@pytest.mark.parametrize("T,topk,E,H,I", [(16, 64, 64, 128, 128),      # the longest routing: 1024 entries, passes of four
                                          (16, 32, 512, 128, 128),     # 512 experts, passes of two
                                          (1, 64, 200, 256, 128),
                                          (1, 2, 3, 6272, 128), (3, 2, 8, 6272, 256)])   # two output tiles a workgroup
def test_moe_decode_workgroup_shapes(fmt, T, topk, E, H, I):
    g = np.random.default_rng(2550 + T + topk)
    L = Layer(2551, fmt, E, H, I)
    x, ids = synth.normal_bf16(g, (T, H)), _ids(g, T, topk, E)
    w = (g.random((T, topk)) / topk).astype(np.float32)
    say(f"[moe decode shapes] {fmt} T={T} topk={topk} E={E} H={H} I={I}")
    got, ref = L.run(x, ids, w), L.ref(x, ids, w)
    _check(got, ref, L.bound(x, ids, w), "layer")
    check_float(got, ref, "layer", rounding_floor=True)


def test_moe_decode_long_lists():
    """More than 64 (pass, K unit) items to a wave of the down launch."""
    g = np.random.default_rng(2560)
    T, topk, E, H, I = 16, 8, 8, 2176, 4352
    L = Layer(2561, "int4_g128", E, H, I)
    x, ids, w = synth.normal_bf16(g, (T, H)), _ids(g, T, topk, E), g.random((T, topk)).astype(np.float32)
    check_float(L.run(x, ids, w), L.ref(x, ids, w), "long lists")


def test_moe_decode_experts_past_4_gib():
    """Expert offsets past 2^32 bytes: only the first and the last expert of 160 hold weights."""
    E, H, I, fmt = 160, 7168, 2048, "int8"
    desc, last = FORMATS[fmt][0], E - 1
    L = Layer(2570, fmt, 2, H, I)
    gu = torch.empty(hq.hq_decode_prepacked_bytes(desc, E, 2 * I, H), dtype=torch.uint8, device=DEV)
    dn = torch.empty(hq.hq_decode_prepacked_bytes(desc, E, H, I), dtype=torch.uint8, device=DEV)
    assert gu.numel() > 2 ** 32
    for whole, two in ((gu, L.gu_dev), (dn, L.dn_dev)):
        n = two.numel() // 2
        assert whole.numel() == E * n
        whole[:n], whole[last * n:] = two[:n], two[n:]
    g = np.random.default_rng(2571)
    for T in (1, 3):
        x, w = synth.normal_bf16(g, (T, H)), g.random((T, 2)).astype(np.float32)
        ids = np.array([[last, 0], [0, -1], [last, last]], np.int32)[:T]
        ref = L.ref(x, np.where(ids == last, 1, ids), w)
        L2 = Layer.__new__(Layer)
        L2.fmt, L2.desc, L2.E, L2.H, L2.I, L2.gu_dev, L2.dn_dev = fmt, desc, E, H, I, gu, dn
        check_float(L2.run(x, ids, w), ref, f"past 4 GiB T={T}")


def test_moe_decode_agrees_with_the_five_calls():
    """The five-call layer on the same packed weights: both are within their roundings of the exact
    layer. The chain rounds four tensors to bf16, half a step (2^-8 of each value) at most each."""
    g = np.random.default_rng(2600)
    E, H, I, topk = 8, 512, 256, 4
    L = Layer(2601, "int4_g128", E, H, I)
    for T in (1, 6, 16):
        x = synth.normal_bf16(g, (T, H))
        ids, w = _ids(g, T, topk, E), g.random((T, topk)).astype(np.float32)
        bm = 16
        cap = hq.hq_moe_align_capacity(T, topk, E, bm)
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
        sid, be, eo, npad = i32(cap), i32(cap // bm), i32(E + 1), i32(1)
        wsb = hq.hq_moe_align_workspace_bytes(T, topk, E, bm)
        ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=DEV)
        dids, dw, dx = to_dev(ids), to_dev(w), to_dev(x.view(np.int16))
        hq.hq_moe_align(dids, T, topk, E, bm, sid, be, eo, npad, ws, wsb)
        b16 = lambda *s: torch.empty(s, dtype=torch.int16, device=DEV)  # noqa: E731
        gu, act, dn, out = b16(T * topk, 2 * I), b16(T * topk, I), b16(T * topk, H), b16(T, H)
        for (t, k, N, K, a, wd, wt, y) in ((T, topk, 2 * I, H, dx, L.gu_dev, None, gu), (T * topk, 1, H, I, act, L.dn_dev, dw, dn)):
            gws = hq.hq_moe_gemm_workspace_bytes(L.desc, t, k, E, N, K, bm)
            wsg = torch.empty(max(gws, 16), dtype=torch.uint8, device=DEV)
            if y is dn:
                hq.hq_moe_silu_mul(T * topk, I, gu, act)
            hq.hq_moe_grouped_gemm(L.desc, t, k, E, N, K, a, None, wd, sid, be, npad, bm, wt, y, wsg, gws)
        hq.hq_moe_combine(T, topk, E, H, dids, dn, out)
        torch.cuda.synchronize()
        ref = L.ref(x, ids, w)
        chain, own = bf16_to_f64(_bits(out)), bf16_to_f64(L.run(x, ids, w))
        e_chain, e_own = np.linalg.norm(chain - ref), np.linalg.norm(own - ref)
        say(f"  T={T}: distance from exact: five calls {e_chain:.3e}, hq_moe_decode {e_own:.3e}")
        assert e_own <= e_chain


# ---- streams, graphs, the step as a whole -----------------------------------------------------
@pytest.mark.parametrize("T", [3, 16])
def test_other_stream_and_graph(T):
    """On a stream of its own, and captured: replayed with new inputs, eager work between the replays."""
    g = np.random.default_rng(2700)
    E, H, I, topk = 16, 256, 768, 4      # the down launch splits its items
    L = Layer(2701, "uint4_g32", E, H, I)
    sh = random_weights(g, "uint4_g32", 2 * I, H)
    sh_dev = to_dev(prepack_host(L.desc, sh, 2 * I, H))
    x = torch.zeros((T, H), dtype=torch.int16, device=DEV)
    logits = torch.zeros((T, E), dtype=torch.float32, device=DEV)
    ids = torch.zeros((T, topk), dtype=torch.int32, device=DEV)
    w = torch.zeros((T, topk), dtype=torch.float32, device=DEV)
    out, act = torch.zeros((T, H), dtype=torch.int16, device=DEV), torch.zeros((T, I), dtype=torch.int16, device=DEV)
    n = hq.hq_moe_decode_workspace_bytes(L.desc, T, topk, E, H, I)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)

    def step(stream=None):
        hq.hq_moe_route(hq.HQ_SCORE_SOFTMAX, T, E, topk, logits, hq.HQ_LOGITS_FP32, None, 1, 1, 2, True, 1.0, ids, w, stream)
        hq.hq_moe_decode(L.desc, T, topk, E, H, I, x, ids, w, L.gu_dev, L.dn_dev, out, ws, n, stream)
        hq.hq_gemv(L.desc, hq.HQ_GEMV_SILU_MUL, T, 2 * I, H, x, sh_dev, act, stream)

    def new_inputs():
        x.copy_(torch.from_numpy(synth.normal_bf16(g, (T, H)).view(np.int16)))
        logits.copy_(torch.from_numpy(g.normal(0, 2, (T, E)).astype(np.float32)))

    def results():
        torch.cuda.synchronize()
        return [t.cpu().numpy().copy() for t in (ids, w, out, act)]

    s = torch.cuda.Stream()
    new_inputs()
    torch.cuda.synchronize()
    step(s)
    other = results()
    step()
    for a, b in zip(other, results()):
        assert np.array_equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        new_inputs()
        ws.fill_(0x7F)
        graph.replay()
        replayed = results()
        for t in (ids, w, out, act):
            t.zero_()
        step()
        for a, b in zip(replayed, results()):
            assert np.array_equal(a, b)


def test_decode_step():
    """Router, routed experts and a shared expert as one MoE block, against the oracle on the same logits."""
    g = np.random.default_rng(2800)
    E, H, I, topk = 32, 512, 256, 6
    L = Layer(2801, "int4_g64", E, H, I)
    sg, sd = random_weights(g, "int4_g64", 2 * I, H), random_weights(g, "int4_g64", H, I)
    sg_dev, sd_dev = to_dev(prepack_host(L.desc, sg, 2 * I, H)), to_dev(prepack_host(L.desc, sd, H, I))
    for T in (1, 4, 16):
        x = synth.normal_bf16(g, (T, H))
        l = route_case(g, T, E, False)
        l[0, 3:] = -np.inf                                  # three experts left for six slots
        bias = g.normal(0, 0.1, E).astype(np.float32)
        ids, w = _route(l, bias, "sigmoid", topk, False, n_group=4, topk_group=2, scale=2.5)
        want_ids, want_w = oracle.ref_route(l.astype(np.float64), bias, "sigmoid", topk, 4, 2, scale=2.5)
        assert np.array_equal(ids, want_ids) and (ids[0, 3:] == -1).all()
        routed = L.run(x, ids, w)
        check_float(routed, L.ref(x, want_ids, want_w), f"routed T={T}", rounding_floor=True)
        act = _gemv(L.desc, True, x, sg_dev, 2 * I, H)
        shared = _gemv(L.desc, False, act, sd_dev, H, I)
        check_float(shared, oracle.ref_gemv(act, dequant(sd, "int4_g64"), False), f"shared T={T}", rounding_floor=True)


def test_two_streams_at_once():
    """Two calls in flight with a workspace each."""
    g = np.random.default_rng(2900)
    L = Layer(2901, "int4_g128", 16, 512, 768)
    calls = []
    for k in range(2):
        x, ids, w = synth.normal_bf16(g, (4, 512)), _ids(g, 4, 4, 16), g.random((4, 4)).astype(np.float32)
        n = hq.hq_moe_decode_workspace_bytes(L.desc, 4, 4, 16, 512, 768)
        calls.append(dict(want=L.run(x, ids, w), x=to_dev(x.view(np.int16)), ids=to_dev(ids), w=to_dev(w), n=n,
                          ws=torch.empty(n, dtype=torch.uint8, device=DEV), out=torch.empty((4, 512), dtype=torch.int16, device=DEV),
                          stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c in calls:
            hq.hq_moe_decode(L.desc, 4, 4, 16, 512, 768, c["x"], c["ids"], c["w"], L.gu_dev, L.dn_dev, c["out"], c["ws"], c["n"], c["stream"])
    torch.cuda.synchronize()
    for c in calls:
        assert np.array_equal(_bits(c["out"]), c["want"])


@pytest.mark.parametrize("fmt,T", [("int4_g32", 1), ("uint4_g128", 4), ("mxfp4", 16), ("int8", 3)])
def test_nothing_is_kept_between_calls(fmt, T):
    """Every buffer overwritten in place between two calls, weights too: the second call's results are those
    of fresh buffers, and every expert that is routed to counts."""
    g = np.random.default_rng(3000 + T)
    E, H, I, topk = 6, 384, 256, 3
    one, two = Layer(3001, fmt, E, H, I), Layer(3002, fmt, E, H, I)
    cases = [(synth.normal_bf16(g, (T, H)), _ids(g, T, topk, E), g.random((T, topk)).astype(np.float32)) for _ in range(2)]
    fresh = two.run(*cases[1])
    n = hq.hq_moe_decode_workspace_bytes(one.desc, T, topk, E, H, I)
    x, ids, w = to_dev(cases[0][0].view(np.int16)), to_dev(cases[0][1]), to_dev(cases[0][2])
    out, ws = torch.zeros((T, H), dtype=torch.int16, device=DEV), torch.zeros(n, dtype=torch.uint8, device=DEV)
    gu, dn = one.gu_dev.clone(), one.dn_dev.clone()

    def moe():
        hq.hq_moe_decode(one.desc, T, topk, E, H, I, x, ids, w, gu, dn, out, ws, n)
        torch.cuda.synchronize()
        return _bits(out).copy()

    assert np.array_equal(moe(), one.run(*cases[0]))
    for old, new in zip((x, ids, w), (cases[1][0].view(np.int16), cases[1][1], cases[1][2])):
        old.copy_(torch.from_numpy(new))
    gu.copy_(two.gu_dev), dn.copy_(two.dn_dev)
    assert np.array_equal(moe(), fresh)
    # an expert's weights zeroed in place: exactly the tokens routed to it change
    per = dn.numel() // E
    for e in range(E):
        kept = dn[e * per:(e + 1) * per].clone()
        dn[e * per:(e + 1) * per] = 0
        got = moe()
        dn[e * per:(e + 1) * per] = kept
        hit = (cases[1][1] == e).any(1)
        assert np.array_equal((got != fresh).any(1), hit), e
    a, b = (prepack_host(one.desc, random_weights(g, fmt, H, H), H, H) for _ in range(2))
    packed, y = to_dev(a), torch.zeros((T, H), dtype=torch.int16, device=DEV)
    for bits in (a, b):
        packed.copy_(torch.from_numpy(bits))
        hq.hq_gemv(one.desc, hq.HQ_GEMV_LINEAR, T, H, H, x, packed, y)
        torch.cuda.synchronize()
        assert np.array_equal(_bits(y), _gemv(one.desc, False, cases[1][0], to_dev(bits), H, H))
