"""GPU parity of the paged 8-bit cache: the append bit for bit with the oracle, the attention over it against float64 within
bounds derived from its arithmetic, and decode steps and prompts built from both with the norm and the products around them."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_prepacked_amd as hq
import synth

from gpu_harness import BF16_NAN_BITS, DEV, bf16_to_f64, say, to_dev
from layer_harness import KV, check_attention, kv_case, normal_rows

pytestmark = pytest.mark.gpu

PAD = 256


# ---- append -----------------------------------------------------------------------------------
def _device(c):
    return {k: to_dev(c[k]) for k in ("cu", "lens", "table", "k_pages", "v_pages", "k_scales", "v_scales")}


def _append(c, d, k, v, max_new=None, stream=None):
    hq.hq_kv_append(c["desc"], c["B"], c["T"], c["max_new"] if max_new is None else max_new, k, v, k.stride(0), d["cu"], d["lens"], d["table"],
                    c["table"].shape[1], d["k_pages"], d["v_pages"], d["k_scales"], d["v_scales"], stream=stream)


def _check_append(c, k, v, max_new=None):
    """k, v: bf16 bits [T, H, D], passed as columns of a wider tensor, as a fused projection leaves them."""
    T, H, D = k.shape
    wide = torch.full((T, 3 * H, D), 1.5, dtype=torch.bfloat16, device=DEV)
    wide[:, H:2 * H] = to_dev(k.view(np.int16)).view(torch.bfloat16)
    wide[:, 2 * H:] = to_dev(v.view(np.int16)).view(torch.bfloat16)
    d = _device(c)
    _append(c, d, wide[:, H:2 * H], wide[:, 2 * H:], max_new)
    torch.cuda.synchronize()
    for what, x in (("k", k), ("v", v)):
        pages, scales = oracle.ref_kv_append(c["fmt"], x, what == "v", c["cu"], c["lens"], c["table"], c[what + "_pages"], c[what + "_scales"], max_new)
        assert np.array_equal(d[what + "_scales"].cpu().numpy(), scales, equal_nan=True), what + " scales"
        got = d[what + "_pages"].cpu().numpy()
        bad = np.argwhere(got != pages)
        assert len(bad) == 0, f"{what}: {len(bad)} codes differ, first at {bad[0]}"
    return d


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("H,D,P", [(1, 64, 16), (3, 96, 32), (8, 128, 16), (2, 128, 64), (2, 192, 128), (1, 256, 256), (5, 64, 256)])
def test_append_matches_oracle(fmt, H, D, P):
    """Pages begun, continued, grown (one token in eight is far larger than the pages' own scale allows), ended inside and on a
    border; single tokens and prompts; sequences without new tokens."""
    g = np.random.default_rng([H, D, P])
    new = [1, 1, 1, 0, 2, 5, P, P + 1, 2 * P + 3, 1, 3]
    lens = [1, P, P + 1, 7, P + 1, P + 2, P, 2 * P, 4 * P + 1, 3 * P - 1, 3]
    c = kv_case(g, fmt, H, D, P, new, lens, peaky=0.01, behind=3)
    k, v = normal_rows(g, c["T"], H, D), normal_rows(g, c["T"], H, D)
    k[::8] = synth.bf16_bits(30 * synth.bf16_bits_to_f32(k[::8]))
    say(f"[append {fmt}] H={H} D={D} P={P}")
    _check_append(c, k, v)


@pytest.mark.parametrize("fmt", list(KV))
def test_append_zeros_and_non_finite(fmt):
    g = np.random.default_rng(2)
    c = kv_case(g, fmt, 2, 64, 16, [4, 4, 1, 1, 1, 1], [4, 20, 5, 6, 7, 18])
    x = normal_rows(g, c["T"], 2, 64)
    x[0:4] = 0                                   # a page of zeros
    x[4, 0, 3], x[5, 1, 5], x[6, 0, 9], x[7, 1, 11] = 0x7FC0, 0xFFFF, 0x7F80, 0xFF80
    x[8] = 0x7FC0                                # a token of NaN alone
    x[9] = 0x8000                                # negative zeros
    x[10, 0] = synth.bf16_bits(np.full(64, 1e-39, np.float32))       # subnormal
    for name in ("k_scales", "v_scales"):        # pages that have held zeros only
        c[name][c["table"][2, 0]] = 0
        c[name[0] + "_pages"][c["table"][2, 0]] = 0
    _check_append(c, x, x[::-1].copy())


@pytest.mark.parametrize("fmt", list(KV))
def test_append_token_by_token(fmt):
    """A sequence written one token at a time over three pages, tokens of growing size among them: every step as the oracle's."""
    g = np.random.default_rng(3)
    c = kv_case(g, fmt, 2, 64, 16, [1], [40])
    c["cu"], c["T"], c["max_new"] = np.array([0, 1], np.int32), 1, 1
    grow = synth.bf16_bits_to_f32(normal_rows(g, 40, 2, 64)) * np.ldexp(1.0, g.integers(-20, 20, (40, 1, 1)))
    x = synth.bf16_bits(grow.astype(np.float32))
    for n in range(1, 41):
        c["lens"] = np.array([n], np.int32)
        d = _check_append(c, x[n - 1:n], x[40 - n:41 - n])
        for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
            c[name] = d[name].cpu().numpy()


@pytest.mark.parametrize("fmt", list(KV))
def test_append_left_out(fmt):
    """Sequences and pages that the arrays make impossible: nothing of them is stored, the others are."""
    g = np.random.default_rng(4)
    c = kv_case(g, fmt, 2, 64, 16, [3, 2, 20, 2, 2, 2], [30, 20, 40, 33, 18, 1])
    k, v = normal_rows(g, c["T"], 2, 64), normal_rows(g, c["T"], 2, 64)
    c["table"][0, 1] = c["desc"].num_pages        # no such page
    c["table"][3, 1] = -1
    c["table"][3, 2] = -2 ** 31
    c["lens"][1] = c["table"].shape[1] * 16 + 1
    _check_append(c, k, v)                        # (sequence 5: two new tokens, one position)
    _check_append(c, k, v, max_new=19)            # sequence 2 has 20
    c["lens"][4] = -1
    c["cu"] = np.array([0, -1, 5, 25, 24, 40, 31], np.int32)
    _check_append(c, k, v)


def test_append_pages_past_32_bits():
    """A cache of more than 4 GiB of codes: the first and the last pages."""
    P, H, D, pages = 256, 8, 128, 20000
    desc = hq.make_kv_desc(hq.HQ_KV_INT8, H, D, P, pages)
    assert hq.hq_kv_cache_bytes(desc) > 1 << 32
    g = np.random.default_rng(5)
    kp = torch.zeros((pages, H, P, D), dtype=torch.uint8, device=DEV)
    vp = torch.zeros((pages, H, D, P), dtype=torch.uint8, device=DEV)
    ks, vs = torch.zeros((pages, H), device=DEV), torch.zeros((pages, H), device=DEV)
    table = np.array([[pages - 1, 0], [pages - 2, 16385]], np.int32)
    new, lens, cu = [300, 257], np.array([300, 257], np.int32), np.array([0, 300, 557], np.int32)
    k, v = normal_rows(g, 557, H, D), normal_rows(g, 557, H, D)
    dk, dv = (to_dev(a.view(np.int16)).view(torch.bfloat16) for a in (k, v))
    dcu, dlens, dtable = to_dev(cu), to_dev(lens), to_dev(table)
    hq.hq_kv_append(desc, 2, 557, 300, dk, dv, H * D, dcu, dlens, dtable, 2, kp, vp, ks, vs)
    small = {int(p): i for i, p in enumerate(table.ravel())}
    at = torch.from_numpy(table.ravel().astype(np.int64)).to(DEV)
    mapped = np.vectorize(small.get)(table).astype(np.int32)
    for x, full, scales, is_value in ((k, kp, ks, False), (v, vp, vs, True)):
        shape = (4, H, D, P) if is_value else (4, H, P, D)
        want, ws = oracle.ref_kv_append("int8", x, is_value, cu, lens, mapped, np.zeros(shape, np.uint8), np.zeros((4, H), np.float32))
        assert np.array_equal(full[at].cpu().numpy(), want) and np.array_equal(scales[at].cpu().numpy(), ws)
        assert int(torch.count_nonzero(scales)) == 4 * H
    # and the attention reads them there
    q = normal_rows(g, 2, H, D)
    qcu = np.array([0, 1, 2], np.int32)
    out = torch.empty((2, H, D), dtype=torch.bfloat16, device=DEV)
    n = hq.hq_attention_workspace_bytes(desc, 2, 2, H, 1, 300)
    hq.hq_attention(desc, 2, 2, H, 1, 300, to_dev(q.view(np.int16)).view(torch.bfloat16), H * D, to_dev(qcu), dlens, dtable, 2, kp, vp, ks, vs, 0.1, 0, out,
                    torch.empty(max(n, 1), dtype=torch.uint8, device=DEV), n)
    torch.cuda.synchronize()
    parts = [t[at].cpu().numpy() for t in (kp, vp, ks, vs)]
    ref = oracle.ref_attention("int8", q, qcu, lens, mapped, *parts, 0.1, 0, np.zeros((2, H, D)))
    check_attention(out.double().cpu().numpy(), *ref, D, 300, "past 32 bits", say)


# ---- attention --------------------------------------------------------------------------------
def _attend(c, d, q, Hq, window=0, sm=None, max_kv=None, max_q=None, ws=None, out=None, stream=None):
    D, T = c["D"], c["T"]
    max_q = c["max_new"] if max_q is None else max_q
    max_kv = int(c["lens"].max()) if max_kv is None else max_kv
    n = hq.hq_attention_workspace_bytes(c["desc"], c["B"], T, Hq, max_q, max_kv)
    if ws is None:
        ws = torch.full((n + 1,), 0xFF, dtype=torch.uint8, device=DEV)      # NaN, were it read
    if out is None:
        out = torch.full((T * Hq * D + PAD,), BF16_NAN_BITS, dtype=torch.int16, device=DEV)
    hq.hq_attention(c["desc"], c["B"], T, Hq, max_q, max_kv, q, q.stride(0), d["cu"], d["lens"], d["table"], c["table"].shape[1], d["k_pages"], d["v_pages"],
                    d["k_scales"], d["v_scales"], D ** -0.5 if sm is None else sm, window, out[:T * Hq * D], ws, n, stream=stream)
    torch.cuda.synchronize()
    assert bool((out[T * Hq * D:] == BF16_NAN_BITS).all()), "written behind the output"
    return out[:T * Hq * D].view(T, Hq, D).cpu().numpy().view(np.uint16)


SENTINEL = 1e300


def _check(c, q, window=0, sm=None, max_kv=None, max_q=None, what=""):
    """q: bf16 bits [T, Hq, D], passed as columns of a wider tensor."""
    T, Hq, D = q.shape
    max_q = c["max_new"] if max_q is None else max_q
    wide = torch.full((T, Hq + 4, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 2:2 + Hq] = to_dev(q.view(np.int16)).view(torch.bfloat16)
    got = _attend(c, _device(c), wide[:, 2:2 + Hq], Hq, window, sm, max_kv, max_q)
    ref = oracle.ref_attention(c["fmt"], q, c["cu"], c["lens"], c["table"], c["k_pages"], c["v_pages"], c["k_scales"], c["v_scales"],
                               D ** -0.5 if sm is None else sm, window, np.full(q.shape, SENTINEL), max_q)
    left = ref[0][:, 0, 0] == SENTINEL
    assert (got[left] == BF16_NAN_BITS).all(), "rows that are left out were written"
    vals = bf16_to_f64(got)
    assert (vals[~left][ref[1][~left].max(-1) == 0] == 0).all(), "rows that see nothing"
    check_attention(vals[~left], *(a[~left] for a in ref), D, int(c["lens"].max()), what or f"{c['fmt']} D={D}", say)


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("H,G,P", [(1, 1, 16), (2, 4, 32), (3, 7, 64), (1, 16, 128), (2, 5, 256), (1, 40, 16)])
def test_single_tokens(fmt, D, H, G, P):
    """One query a sequence: lengths around every border of 16, 64 and pages, and one that is split over workgroups."""
    g = np.random.default_rng([D, H, G, P])
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000, 1025]
    c = kv_case(g, fmt, H, D, P, [1] * len(lens), lens, peaky=0.6)
    _check(c, normal_rows(g, c["T"], H * G, D), what=f"{fmt} D={D} H={H} G={G} P={P}")


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("D,H,G,P,window", [(64, 2, 1, 16, 0), (128, 2, 4, 64, 0), (128, 1, 8, 16, 100), (96, 1, 3, 32, 1), (256, 2, 6, 32, 64), (192, 1, 2, 128, 65),
                                            (128, 4, 2, 256, 1000)])
def test_several_tokens(fmt, D, H, G, P, window):
    """Drafted tokens, whole prompts, pieces of prompts, and sequences without new tokens in one call; masks on every side."""
    g = np.random.default_rng([D, H, G, P, window])
    new = [1, 3, 5, 0, 16, 17, 64, 65, 130, 1, 2, 200]
    lens = [1, 3, 70, 50, 16, 400, 64, 65, 130, 700, 129, 333]
    c = kv_case(g, fmt, H, D, P, new, lens, peaky=0.6, behind=2)
    _check(c, normal_rows(g, c["T"], H * G, D), window=window, what=f"{fmt} D={D} H={H} G={G} P={P} window={window}")


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("H,G,P,new,length,window", [(1, 4, 16, 256, 256, 0), (2, 8, 64, 129, 129, 0), (1, 16, 256, 70, 1000, 0), (1, 5, 32, 333, 700, 100),
                                                     (2, 64, 16, 17, 65, 0), (1, 128, 128, 9, 640, 33), (1, 8, 16, 200, 90, 0)])
def test_many_rows_of_one_long_sequence(fmt, H, G, P, new, length, window):
    """More rows than a workgroup of 128 or 256 takes, a broken last tile, more tokens than positions; max_kv says that the past may be
    long, whatever it is."""
    g = np.random.default_rng([H, G, P, new])
    c = kv_case(g, fmt, H, 128, P, [new], [length], peaky=0.6, behind=1)
    if length == 700:
        c["table"][0, 3], c["table"][0, 15] = -1, c["desc"].num_pages      # pages freed behind a window, and one in it
    _check(c, normal_rows(g, c["T"], H * G, 128), window=window, max_kv=4096, what=f"{fmt} H={H} G={G} P={P} {new} on {length}")


@pytest.mark.parametrize("H,G,D,max_kv", [(2, 1, 64, None), (1, 8, 128, 4096)])
def test_widest_window(H, G, D, max_kv):
    """The largest window there is, with more new tokens than positions: differences of the two leave 32 bits."""
    g = np.random.default_rng(23)
    c = kv_case(g, "fp8", H, D, 16, [4, 200, 40, 300], [2, 90, 40, 200], peaky=0.6)
    _check(c, normal_rows(g, c["T"], H * G, D), window=2 ** 31 - 1, max_kv=max_kv, what=f"widest window D={D}")


@pytest.mark.parametrize("window", [0, 1024])
def test_workspace_does_not_ask_for_the_window(window):
    """43 heads of 300 rows that are told of 4096 positions: more parts with the window's small tiles than without it."""
    g = np.random.default_rng(22)
    c = kv_case(g, "int8", 43, 128, 64, [300], [1500], peaky=0.6)
    _check(c, normal_rows(g, c["T"], 43, 128), window=window, max_kv=4096, what=f"window={window}")


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("H,G,P,window", [(1, 4, 16, 0), (2, 8, 128, 0), (1, 16, 64, 70), (2, 3, 32, 500)])
def test_many_rows_of_several_sequences(fmt, H, G, P, window):
    """Long pieces of several sequences in one call, at both ends of their lengths, with single tokens, an empty sequence and one
    that the arrays make impossible among them."""
    g = np.random.default_rng([H, G, P, window])
    new, lens = [300, 1, 190, 0, 257, 333, 40], [700, 900, 190, 5, 260, 1500, 1100]
    c = kv_case(g, fmt, H, 128, P, new, lens, peaky=0.6, behind=3)
    c["lens"][6] = c["table"].shape[1] * P + 1
    _check(c, normal_rows(g, c["T"], H * G, 128), window=window, max_kv=4096, what=f"{fmt} H={H} G={G} P={P} window={window}")


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("new", [1, 4, 40])
def test_rows_that_see_nothing(fmt, new):
    """Empty sequences, more queries than positions, no page left, pages freed in the middle: rows without a token are zeros, the
    others see what is there."""
    g = np.random.default_rng(new)
    lens = [0, 1, 3, 100, 100, 200, 39, 41]
    c = kv_case(g, fmt, 2, 64, 16, [new] * len(lens), [max(n, 1) for n in lens])
    c["lens"] = np.array(lens, np.int32)
    c["table"][3] = -1
    c["table"][4, 1:4] = c["desc"].num_pages + 5
    c["table"][5, :8] = -2 ** 31
    q = normal_rows(g, c["T"], 6, 64)
    _check(c, q, what=f"{fmt} new={new}")
    _check(c, q, window=20, what=f"{fmt} new={new} window")


@pytest.mark.parametrize("fmt", list(KV))
def test_left_out(fmt):
    g = np.random.default_rng(7)
    c = kv_case(g, fmt, 2, 64, 16, [2, 3, 30, 4, 1], [50, 60, 70, 80, 90])
    q = normal_rows(g, c["T"], 4, 64)
    _check(c, q, max_q=29, max_kv=90)
    c["lens"][1], c["lens"][3] = -5, c["table"].shape[1] * 16 + 1
    _check(c, q, max_kv=90)
    c["cu"] = np.array([0, 2, 1, 35, 39, 41], np.int32)     # (34 rows of sequence 2 are more than max_q)
    _check(c, q, max_kv=90)


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("H,P,max_kv,window", [(64, 16, None, 0), (64, 32, None, 70), (1, 64, 1 << 20, 0)])
def test_seventeen_to_thirty_two_rows(fmt, D, H, P, max_kv, window):
    """Drafted tokens of heads that fill the card, and of one head with a past that may be long: all rows of a head in one workgroup."""
    g = np.random.default_rng([D, H, P])
    c = kv_case(g, fmt, H, D, P, [4, 1, 3, 0, 2, 4, 4], [4, 130, 65, 20, 1, 64, 203], peaky=0.6, behind=1)
    _check(c, normal_rows(g, c["T"], H * 8, D), window=window, max_kv=max_kv, what=f"{fmt} D={D} H={H} P={P} window={window}")


@pytest.mark.parametrize("max_kv", [0, 64, 300, 5000, 1 << 20])
def test_any_number_of_parts(max_kv):
    """max_kv sets how the work is shared out, too small or too large, never what is computed."""
    g = np.random.default_rng(8)
    for new, lens in (([1, 1, 1], [5000, 64, 1]), ([2, 9, 0], [5000, 300, 70])):
        c = kv_case(g, "fp8", 1, 128, 64, new, lens)
        _check(c, normal_rows(g, c["T"], 4, 128), max_kv=max_kv, what=f"max_kv={max_kv} new={new}")


def test_peaked_and_flat():
    """Scores of a size where one token takes all, negative and zero scales, and a flat softmax over a long past."""
    g = np.random.default_rng(9)
    c = kv_case(g, "fp8", 2, 128, 32, [1, 40, 3], [900, 300, 20000])
    q = normal_rows(g, c["T"], 6, 128)
    for sm in (0.0, 1e-3, 0.5, -0.1):
        _check(c, q, sm=sm, what=f"sm_scale {sm}")


def test_bad_queries_alone():
    """NaN or infinity in a query's head: that row alone."""
    g = np.random.default_rng(10)
    for new in (2, 50):
        c = kv_case(g, "fp8", 2, 64, 16, [new, 1], [500, 77])
        q = normal_rows(g, c["T"], 8, 64)
        d = _device(c)
        up = lambda a: to_dev(a.view(np.int16)).view(torch.bfloat16)  # noqa: E731
        want = _attend(c, d, up(q), 8)
        bad = q.copy()
        bad[1, 5, 3], bad[0, 2, 9] = 0x7FC0, 0x7F80
        got = _attend(c, d, up(bad), 8)
        assert np.isnan(bf16_to_f64(got[1, 5])).all()
        same = np.ones((c["T"], 8), bool)
        same[1, 5] = same[0, 2] = False
        assert np.array_equal(got[same], want[same])


def test_bad_keys_reach_who_sees_them():
    """A NaN key (as the append stores it): rows before it, and rows whose window has passed it, do not notice."""
    g = np.random.default_rng(11)
    for new in (4, 40):
        c = kv_case(g, "fp8", 1, 64, 16, [new], [200])
        at = 198 if new == 4 else 170
        c["k_pages"][c["table"][0, at // 16], 0, at % 16, 5] = 0x7F
        q = normal_rows(g, new, 4, 64)
        got = bf16_to_f64(_attend(c, _device(c), to_dev(q.view(np.int16)).view(torch.bfloat16), 4, window=10))
        pos = 200 - new + np.arange(new)
        sees = (at <= pos) & (at > pos - 10)
        assert np.isnan(got[sees]).all() and np.isfinite(got[~sees]).all() and sees.any() and (~sees).any()


@pytest.mark.parametrize("fmt", list(KV))
def test_bad_queries_and_keys_among_many_rows(fmt):
    """NaN and infinity in two query rows of a long piece, then a NaN key in its middle: every other row keeps its bits."""
    g = np.random.default_rng(24)
    c = kv_case(g, fmt, 1, 128, 64, [300], [700])
    q = normal_rows(g, 300, 4, 128)
    up = lambda a: to_dev(a.view(np.int16)).view(torch.bfloat16)  # noqa: E731
    clean = _attend(c, _device(c), up(q), 4, max_kv=4096)
    assert np.isfinite(bf16_to_f64(clean)).all()
    bad = q.copy()
    bad[17, 1, 5], bad[100, 3, 0] = 0x7FC0, 0x7F80
    got = _attend(c, _device(c), up(bad), 4, max_kv=4096)
    others = np.ones((300, 4), bool)
    others[17, 1] = others[100, 3] = False
    assert np.array_equal(got[others], clean[others]) and np.isnan(bf16_to_f64(got[17, 1])).all() and not np.isfinite(bf16_to_f64(got[100, 3])).all()
    if fmt == "fp8":
        c["k_pages"][c["table"][0, 500 // 64], 0, 500 % 64, 77] = 0x7F
        got = _attend(c, _device(c), up(q), 4, max_kv=4096)
        sees = 400 + np.arange(300) >= 500
        assert np.isnan(bf16_to_f64(got[sees])).all() and np.array_equal(got[~sees], clean[~sees])


def test_pages_that_sequences_share():
    """A prefix held once: the first pages of three sequences are the same, the sequences' own follow."""
    g = np.random.default_rng(25)
    for D, new, lens in ((64, [1, 40, 3], [130, 200, 70]), (128, [300, 1, 280], [500, 77, 400])):
        c = kv_case(g, "int8", 2, D, 64, new, lens, peaky=0.6)
        c["table"][1:, 0] = c["table"][0, 0]
        _check(c, normal_rows(g, c["T"], 8, D), max_kv=4096, what=f"shared pages D={D}")


def test_nothing_behind_the_end_is_read():
    """The slots behind a sequence's end hold NaN codes, the other pages NaN scales (kv_case); so do, here, freed pages."""
    g = np.random.default_rng(12)
    c = kv_case(g, "fp8", 2, 128, 64, [1, 20], [130, 90])
    q = normal_rows(g, c["T"], 4, 128)
    _check(c, q, window=30)
    c["table"][0, 0], c["table"][1, 0] = -1, -1           # behind the window of every row of sequence 0, inside some of 1's
    _check(c, q, window=30)


def test_out_may_be_q():
    g = np.random.default_rng(13)
    for new, lens in (([1, 1], [300, 3000]), ([100, 3], [100, 500])):
        c = kv_case(g, "int8", 2, 64, 16, new, lens)
        q = normal_rows(g, c["T"], 4, 64)
        d = _device(c)
        want = _attend(c, d, to_dev(q.view(np.int16)).view(torch.bfloat16), 4)
        both = torch.cat([to_dev(q.view(np.int16)).ravel(), torch.full((PAD,), BF16_NAN_BITS, dtype=torch.int16, device=DEV)])
        n = c["T"] * 4 * 64
        got = _attend(c, d, both[:n].view(c["T"], 4, 64).view(torch.bfloat16), 4, out=both)
        assert np.array_equal(got, want)


def test_same_bits_every_time():
    """No order of workgroups enters: the same call again, and with other work on the card."""
    g = np.random.default_rng(14)
    c = kv_case(g, "int8", 2, 128, 16, [1, 1, 5, 70], [9000, 4, 2000, 600])
    q = to_dev(normal_rows(g, c["T"], 8, 128).view(np.int16)).view(torch.bfloat16)
    d = _device(c)
    want = _attend(c, d, q, 8)
    side, noise = torch.cuda.Stream(), torch.randn((2048, 2048), device=DEV)
    for _ in range(5):
        with torch.cuda.stream(side):
            for _ in range(3):
                noise = (noise @ noise).clamp(-1, 1)
        assert np.array_equal(_attend(c, d, q, 8), want)


# ---- a run of them together -------------------------------------------------------------------
def test_layer_prompt_and_decode_in_graphs():
    """A layer's attention block on two sequences: norm -> packed projection -> append -> attention, a prompt first, then decode
    steps replayed from one captured graph, with each step's results against the oracle run on the same codes."""
    g = np.random.default_rng(15)
    B, H, G, D, P, hidden = 2, 2, 4, 64, 16, 512
    Hq, width, pages = H * G, (H * G + 2 * H) * D, 20
    desc, kv = hq.DESC_W8A8, hq.make_kv_desc(hq.HQ_KV_FP8_E4M3, H, D, P, pages)
    w8 = g.integers(-127, 128, (width, hidden), dtype=np.int64).astype(np.int8)
    sw = np.full(width, 1 / 1500, np.float32)
    packed = np.zeros(hq.hq_prepacked_bytes(desc, 1, width, hidden), np.uint8)
    hq.hq_prepack_weights(desc, 1, width, hidden, w8, sw, None, packed)
    wp, wnorm = to_dev(packed), synth.bf16_bits(g.uniform(0.5, 1.5, hidden).astype(np.float32))
    dw = to_dev(wnorm.view(np.int16)).view(torch.bfloat16)
    table = np.arange(pages, dtype=np.int32).reshape(B, -1)[:, ::-1].copy()
    cache = {"k_pages": np.full((pages, H, P, D), 0xFF, np.uint8), "v_pages": np.full((pages, H, D, P), 0xFF, np.uint8),
             "k_scales": np.full((pages, H), np.nan, np.float32), "v_scales": np.full((pages, H), np.nan, np.float32)}
    dc, dtable = {k: to_dev(v) for k, v in cache.items()}, to_dev(table)

    def buffers(T, max_q, max_kv):
        n = hq.hq_attention_workspace_bytes(kv, B, T, Hq, max_q, max_kv)
        n2 = hq.hq_gemm_workspace_bytes(desc, T, width, hidden)
        e = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
        return {"x": e(T, hidden), "r": e(T, hidden), "q8": e(T, hidden, t=torch.int8), "s": e(T, t=torch.float32), "qkv": e(T, Hq + 2 * H, D),
                "out": e(T, Hq, D), "cu": e(B + 1, t=torch.int32), "lens": e(B, t=torch.int32), "ws": e(n + 1, t=torch.uint8), "n": n,
                "ws2": e(n2 + 1, t=torch.uint8), "n2": n2, "T": T, "max_q": max_q, "max_kv": max_kv}

    def step(b, stream=None):
        T, k, v = b["T"], b["qkv"][:, Hq:Hq + H], b["qkv"][:, Hq + H:]
        hq.hq_rms_norm(hq.HQ_ACT_INT8_PER_TOKEN, T, hidden, b["x"], b["r"], dw, 1e-6, b["r"], b["q8"], b["s"], stream=stream)
        hq.hq_gemm(desc, T, width, hidden, b["q8"], b["s"], wp, b["qkv"], b["ws2"], b["n2"], stream=stream)
        hq.hq_kv_append(kv, B, T, b["max_q"], k, v, width, b["cu"], b["lens"], dtable, table.shape[1], *(dc[n] for n in cache), stream=stream)
        hq.hq_attention(kv, B, T, Hq, b["max_q"], b["max_kv"], b["qkv"][:, :Hq], width, b["cu"], b["lens"], dtable, table.shape[1], *(dc[n] for n in cache),
                        D ** -0.5, 0, b["out"], b["ws"], b["n"], stream=stream)

    def set_inputs(b, new, lens):
        x, r = synth.normal_bf16(g, (b["T"], hidden)), synth.normal_bf16(g, (b["T"], hidden))
        b["x"].copy_(to_dev(x.view(np.int16)).view(torch.bfloat16))
        b["r"].copy_(to_dev(r.view(np.int16)).view(torch.bfloat16))
        b["cu"].copy_(to_dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
        b["lens"].copy_(to_dev(np.array(lens, np.int32)))
        return x, r

    def check(b, x, r, what):
        torch.cuda.synchronize()
        h, v = oracle.ref_rms_norm(x, r, wnorm, 1e-6)
        codes, s = oracle.quantize_values(v, "int8")
        assert np.array_equal(b["q8"].cpu().numpy(), codes) and np.array_equal(b["s"].cpu().numpy(), s)
        assert np.array_equal(b["r"].view(torch.int16).cpu().numpy().view(np.uint16), h)
        _, _, y = oracle.ref_w8a8(codes, s, w8, sw)
        qkv = b["qkv"].view(torch.int16).cpu().numpy().view(np.uint16)
        y = oracle.decode_bf16(y) if y.dtype == np.uint16 else y
        assert np.allclose(bf16_to_f64(qkv.reshape(b["T"], -1)), y, rtol=2.0 ** -7, atol=1e-30)
        cu, lens = b["cu"].cpu().numpy(), b["lens"].cpu().numpy()
        for n, at in (("k", Hq), ("v", Hq + H)):
            cache[n + "_pages"], cache[n + "_scales"] = oracle.ref_kv_append("fp8", qkv[:, at:at + H], n == "v", cu, lens, table, cache[n + "_pages"], cache[n + "_scales"])
            assert np.array_equal(dc[n + "_pages"].cpu().numpy(), cache[n + "_pages"])
            assert np.array_equal(dc[n + "_scales"].cpu().numpy(), cache[n + "_scales"], equal_nan=True)
        ref = oracle.ref_attention("fp8", qkv[:, :Hq], cu, lens, table, *(cache[n] for n in cache), D ** -0.5, 0, np.zeros((b["T"], Hq, D)))
        check_attention(bf16_to_f64(b["out"].view(torch.int16).cpu().numpy().view(np.uint16)), *ref, D, int(lens.max()), what, say)

    new = [70, 21]
    prompt = buffers(sum(new), max(new), 160)
    lens = list(new)
    io = set_inputs(prompt, new, lens)
    step(prompt)
    check(prompt, *io, "prompt")

    one = buffers(B, 1, 160)
    set_inputs(one, [1, 1], lens)      # (lengths unchanged: writes the prompts' last tokens anew)
    one["lens"].fill_(0)               # nothing to store, nothing to see
    step(one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(one)
    for k in range(14):
        lens = [n + 1 for n in lens]
        io = set_inputs(one, [1, 1], lens)
        graph.replay()
        check(one, *io, f"decode step {k}")
    side = torch.cuda.Stream()
    lens = [n + 1 for n in lens]
    io = set_inputs(one, [1, 1], lens)
    side.wait_stream(torch.cuda.current_stream())
    step(one, side)
    torch.cuda.current_stream().wait_stream(side)
    check(one, *io, "on another stream")
    # a fork: the pages of a sequence copied, the copy read in its place
    before = one["out"].clone()
    free = to_dev(np.arange(pages, 2 * pages, dtype=np.int32).reshape(B, -1))
    twice = {n: torch.cat([t, t.clone()]) for n, t in dc.items()}
    for n in ("k_pages", "v_pages", "k_scales", "v_scales"):
        twice[n][pages:][(free.long() - pages).flatten()] = dc[n][dtable.long().flatten()]
    kv2 = hq.make_kv_desc(hq.HQ_KV_FP8_E4M3, H, D, P, 2 * pages)
    hq.hq_attention(kv2, B, B, Hq, 1, 160, one["qkv"][:, :Hq], width, one["cu"], one["lens"], free, table.shape[1], *(twice[n] for n in cache), D ** -0.5, 0,
                    one["out"], one["ws"], one["n"])
    torch.cuda.synchronize()
    assert bool((one["out"] == before).all())


@pytest.mark.parametrize("fmt", list(KV))
def test_value_scales_far_apart(fmt):
    """Pages whose values are many powers of two apart, pages of zeros (scale 0), keys' scales of 0: weights are rounded relative to
    the row's largest p * scale, wherever that is."""
    g = np.random.default_rng(16)
    for new, lens in (([1, 3], [700, 90]), ([60, 33], [200, 400])):
        c = kv_case(g, fmt, 2, 64, 16, new, lens, peaky=0.8)
        live = ~np.isnan(c["v_scales"])
        for exponents in ((-40, 40), (-3, 3), (-140, -120), (100, 110)):
            d = dict(c)
            d["v_scales"] = np.where(live, np.ldexp(c["v_scales"], g.integers(*exponents, c["v_scales"].shape)), np.nan).astype(np.float32)
            d["k_scales"] = c["k_scales"].copy()
            zero = live & (g.random(live.shape) < 0.2)
            d["v_scales"][zero] = 0
            d["v_pages"] = np.where(zero[:, :, None, None], 0, c["v_pages"]).astype(np.uint8)
            d["k_scales"][live & (g.random(live.shape) < 0.1)] = 0
            _check(d, normal_rows(g, c["T"], 6, 64), what=f"{fmt} scales 2^{exponents}")


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("D,new,length,max_kv", [(64, 1, 1500, None), (128, 4, 1500, None), (128, 40, 700, None), (128, 300, 900, 4096)])
def test_values_of_zero_first(fmt, D, new, length, max_kv):
    """Whole blocks whose values are zero (scale 0) where a row, or a wave's part of it, begins: they count in the sum alone."""
    g = np.random.default_rng([17, D, new])
    for zeros in (slice(0, 8), slice(0, 24), slice(4, None), slice(None)):
        c = kv_case(g, fmt, 2, D, 16, [new], [length], peaky=0.6)
        pages = c["table"][0][c["table"][0] >= 0][zeros]
        c["v_scales"][pages] = 0
        c["v_pages"][pages] = 0
        _check(c, normal_rows(g, new, 8, D), max_kv=max_kv, what=f"{fmt} D={D} new={new} zeros {zeros}")
