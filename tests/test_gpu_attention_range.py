"""Attention over the paged cache at the ends of its number ranges, against float64: values near the largest bf16,
scores of any size, rows most of whose weight is on a token of value 0, and
caches past 4 GiB."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_prepacked_amd as hq

from gpu_harness import DEV, bf16_to_f64, say, to_dev
from layer_harness import KV, check_attention, kv_case, normal_rows
from test_gpu_attention import _attend, _device

pytestmark = pytest.mark.gpu

# (D, G, new, length, max_kv) that take: four waves' join, the split positions' join, 32 rows a workgroup, 128 rows in one part and in
# several, 256 rows in one part and in several
PATHS = [(64, 4, 1, 300, 64), (128, 4, 4, 1500, 1500), (256, 6, 5, 700, 700), (64, 4, 40, 700, 64), (128, 4, 40, 2900, 2900), (96, 3, 50, 2000, 2000),
         (128, 4, 300, 400, 2048), (128, 4, 300, 1300, 4096)]


def _run(c, q, max_kv, sm=None):
    D = c["D"]
    sm = D ** -0.5 if sm is None else sm
    got = bf16_to_f64(_attend(c, _device(c), to_dev(q.view(np.int16)).view(torch.bfloat16), q.shape[1], sm=sm, max_kv=max_kv))
    ref = oracle.ref_attention(c["fmt"], q, c["cu"], c["lens"], c["table"], c["k_pages"], c["v_pages"], c["k_scales"], c["v_scales"], sm, 0, np.zeros(q.shape))
    return got, ref


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("D,G,new,length,max_kv", PATHS)
def test_values_near_the_largest(fmt, D, G, new, length, max_kv):
    """Averages of values whose sums pass fp32's range: all of the largest bf16 (as an infinity is stored), of both signs, and scales up
    to 2^118."""
    g = np.random.default_rng([D, new, length])
    c = kv_case(g, fmt, 2, D, 16, [new], [length], peaky=0.01)
    q = normal_rows(g, new, 2 * G, D)
    largest = float(oracle.decode_bf16(np.array([0x7F7F], np.uint16))[0])
    plain, pages, live = c["v_pages"], c["v_scales"].copy(), ~np.isnan(c["v_scales"])
    top, low = (0x7E, 0xFE) if fmt == "fp8" else (127, 0x81)
    for what in ("largest", "both signs", "far scales"):
        if what == "far scales":
            c["v_pages"] = plain
            c["v_scales"] = np.where(live, np.ldexp(pages, g.integers(100, 124, pages.shape)), np.nan).astype(np.float32)
        else:
            sign = g.random(plain.shape) < (0.5 if what == "both signs" else 0.0)
            c["v_pages"] = np.where(sign, low, top).astype(np.uint8)
            c["v_scales"] = np.where(live, np.float32(largest) * (np.float32(1) / np.float32(448 if fmt == "fp8" else 127)), np.nan).astype(np.float32)
        got, ref = _run(c, q, max_kv)
        check_attention(got, *ref, D, length, f"{fmt} D={D} new={new} on {length}: {what}", say)


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("D,G,new,length,max_kv", PATHS)
def test_scores_of_any_size(fmt, D, G, new, length, max_kv):
    """Scores so large that fp32 tells only the largest apart, with values' scales up to 2^far from their mean: a row is the value of its
    largest score, rounded once. Rows whose two largest are nearer than the scores' rounding (2^-22 (D + 8) of the products' size, each) and
    40 + 2 far log 2 are left out; there are few. So every other weight is at most e^-40 4^-far, `length` of them add up to that many times
    the largest value at most, and 2^-8 (the result), 2^-11 (its weight as an fp16) and 2^-20 (the fp32 steps) of the value itself come on
    top."""
    g = np.random.default_rng([1, D, new, length])
    c = kv_case(g, fmt, 2, D, 16, [new], [length])
    live = ~np.isnan(c["v_scales"])
    sm, at = 0.3, np.arange(length)
    pages = c["table"][0, at // 16]
    val = oracle.decode_e4m3 if fmt == "fp8" else (lambda a: oracle.decode_int8(a.view(np.int8)))
    plain = c["v_scales"]
    for bits, far in ((12, 0), (20, 0), (27, 0), (30, 20), (48, 0), (64, 90), (110, 90)):
        c["v_scales"] = np.where(live, np.ldexp(plain, g.integers(-far, far + 1, plain.shape)), np.nan).astype(np.float32)
        q = normal_rows(g, new, 2 * G, D, 2.0 ** bits)
        got, ref = _run(c, q, max_kv, sm)
        qv, checked, worst = oracle.decode_bf16(q), 0, 0.0
        for h in range(2):
            k = val(c["k_pages"][pages, h, at % 16]) * c["k_scales"][pages, h].astype(np.float64)[:, None]
            v = val(c["v_pages"][pages, h, :, at % 16]) * c["v_scales"][pages, h].astype(np.float64)[:, None]
            s = sm * np.einsum("thd,jd->thj", qv[:, h * G:h * G + G], k)
            s = np.where(at > (length - new + np.arange(new))[:, None, None], -np.inf, s)
            order = np.sort(s, -1)
            sure = order[..., -1] - order[..., -2] > 2 * 2.0 ** -22 * (D + 8) * ref[4][:, h * G:h * G + G] + 40 + 2 * far * np.log(2)
            want, have = v[s.argmax(-1)][sure], got[:, h * G:h * G + G][sure]
            assert np.isfinite(have).all(), f"2^{bits}"
            bound = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20) * np.abs(want) + length * np.exp(-40) * 4.0 ** -far * np.abs(v).max() + 2.0 ** -134
            worst = max([worst, *(np.abs(have - want) / bound).ravel()])
            checked += sure.sum()
        say(f"  {fmt} D={D} new={new} on {length}, q of 2^{bits}: {checked} of {2 * G * new} rows, worst {worst:.3f} of its bound")
        assert worst <= 1.0 and checked >= 0.8 * 2 * G * new, f"2^{bits}"


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("D,G,new,length,max_kv", PATHS)
def test_largest_scores_on_values_of_zero(fmt, D, G, new, length, max_kv):
    """Rows' largest scores of 2^124 to 2^127, and values of zero (scale 0) where a row begins, or everywhere: rows of a value, zeros, nothing else."""
    g = np.random.default_rng([3, D, new, length])
    c = kv_case(g, fmt, 2, D, 16, [new], [length])
    q = normal_rows(g, new, 2 * G, D, 2.0 ** 100)
    sm = 2.0 ** 23 / D ** 0.5
    for zeros in (slice(0, 6), slice(None)):
        c["v_scales"][c["table"][0][c["table"][0] >= 0][zeros]] = 0
        got, ref = _run(c, q, max_kv, sm)
        largest = np.abs(ref[0]).max()
        assert np.isfinite(got).all() and (np.abs(got) <= largest * (1 + 2.0 ** -7)).all(), zeros
        assert zeros != slice(None) or (got == 0).all()


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("D,G,new,length,max_kv", [(64, 4, 1, 30000, 64), (128, 4, 4, 20000, 64), (64, 4, 40, 20000, 64), (128, 2, 40, 9000, 64), (256, 1, 40, 9000, 64),
                                                   (128, 4, 64, 20000, 2048)])
@pytest.mark.parametrize("share", [0.9, 0.99, 0.999])
def test_first_token_takes_the_weight(fmt, D, G, new, length, max_kv, share):
    """A first token with `share` of a row's weight and a value of 0: the row is what the others leave. The result's rounding to bf16, uniform
    within a step of 2^-7 of the binade, is 2^-7 / sqrt(28) of the whole's size (the mean square of 1 .. 2 is 7 / 3); the roundings of
    the weights stay below the same, so that twice that is never passed."""
    g = np.random.default_rng([2, D, new, length])
    c = kv_case(g, fmt, 1, D, 32, [new], [length], peaky=0.3)
    q, sm, first = normal_rows(g, new, G, D), D ** -0.5, c["table"][0, 0]
    q[..., 0] = 0x4200                                 # 32
    c["k_pages"][..., 0] = 0                           # channel 0: the first token's alone
    c["k_pages"][first] = 0
    c["v_pages"][first, :, :, 0] = 0
    c["k_pages"][first, 0, 0, 0] = 0x68 if fmt == "fp8" else 64         # 64
    c["k_scales"][first] = 0
    val = oracle.decode_e4m3 if fmt == "fp8" else (lambda a: oracle.decode_int8(a.view(np.int8)))
    at = np.arange(length)
    page = c["table"][0, at // 32]
    k = val(c["k_pages"][page, 0, at % 32]) * c["k_scales"][page, 0].astype(np.float64)[:, None]
    v = val(c["v_pages"][page, 0, :, at % 32]) * c["v_scales"][page, 0].astype(np.float64)[:, None]
    score = sm * np.einsum("tgd,jd->tgj", oracle.decode_bf16(q), k)
    others = np.log(np.exp(score[0, 0]).sum())
    scale = np.float32((others + np.log(share / (1 - share))) / (sm * 32 * 64))
    c["k_scales"][first] = scale                       # (the first page's other keys are zeros)
    score[..., 0] = sm * 32 * 64 * float(scale)
    weight = np.exp(np.where(at > (length - new + np.arange(new))[:, None, None], -np.inf, score))
    ref = weight @ v / weight.sum(-1, keepdims=True)
    got = bf16_to_f64(_attend(c, _device(c), to_dev(q.view(np.int16)).view(torch.bfloat16), G, sm=sm, max_kv=max_kv))
    error = float(np.linalg.norm(got - ref) / np.linalg.norm(ref))
    say(f"  {fmt} D={D} new={new} on {length}, {share}: {error / (2.0 ** -7 / 28 ** 0.5):.3f} of the rounding to bf16")
    assert error <= 2 * 2.0 ** -7 / 28 ** 0.5


@pytest.mark.parametrize("fmt", list(KV))
def test_many_rows_past_32_bits(fmt):
    """A cache of more than 4 GiB of codes, its first and last pages, read by every kernel: one token, 24 rows, 128 and 256 rows a workgroup."""
    P, H, D, pages = 256, 8, 128, 20000
    desc = hq.make_kv_desc(KV[fmt], H, D, P, pages)
    assert hq.hq_kv_cache_bytes(desc) > 1 << 32
    g = np.random.default_rng(32)
    kp = torch.zeros((pages, H, P, D), dtype=torch.uint8, device=DEV)
    vp = torch.zeros((pages, H, D, P), dtype=torch.uint8, device=DEV)
    ks, vs = torch.zeros((pages, H), device=DEV), torch.zeros((pages, H), device=DEV)
    table = np.array([[pages - 1, 0], [pages - 2, 16385]], np.int32)
    lens, cu = np.array([300, 257], np.int32), np.array([0, 300, 557], np.int32)
    up = lambda a: to_dev(a.view(np.int16)).view(torch.bfloat16)  # noqa: E731
    k, v = normal_rows(g, 557, H, D), normal_rows(g, 557, H, D)
    dlens, dtable = to_dev(lens), to_dev(table)
    hq.hq_kv_append(desc, 2, 557, 300, up(k), up(v), H * D, to_dev(cu), dlens, dtable, 2, kp, vp, ks, vs)
    at = torch.from_numpy(table.ravel().astype(np.int64)).to(DEV)
    parts = [t[at].cpu().numpy() for t in (kp, vp, ks, vs)]
    mapped = np.arange(4, dtype=np.int32).reshape(2, 2)
    for new, max_kv in (([1, 1], 300), ([24, 3], 300), ([40, 200], 300), ([300, 257], 4096)):
        T, most = sum(new), max(new)
        qcu, q = np.array([0, new[0], T], np.int32), normal_rows(g, T, H, D)
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV)
        n = hq.hq_attention_workspace_bytes(desc, 2, T, H, most, max_kv)
        hq.hq_attention(desc, 2, T, H, most, max_kv, up(q), H * D, to_dev(qcu), dlens, dtable, 2, kp, vp, ks, vs, 0.1, 0, out,
                        torch.empty(max(n, 1), dtype=torch.uint8, device=DEV), n)
        torch.cuda.synchronize()
        ref = oracle.ref_attention(fmt, q, qcu, lens, mapped, *parts, 0.1, 0, np.zeros(q.shape))
        check_attention(out.double().cpu().numpy(), *ref, D, 300, f"{fmt} past 32 bits, {new} tokens", say)
