"""CPU checks of the norm, cache and attention calls: oracle pins, what the bounds can see, and every refusal (made on
the host before any launch, so they run without a GPU)."""
import math

import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_prepacked_amd as hq
import synth

from layer_harness import NORM, attention_bounds, kv_case, normal_rows

INV, UNS, WSP = hq.HQ_ERR_INVALID_ARGUMENT, hq.HQ_ERR_UNSUPPORTED, hq.HQ_ERR_WORKSPACE


def _status(f, *a, **k):
    with pytest.raises(hq.HQError) as ei:
        f(*a, **k)
    return ei.value.status


# ---- oracle pins ------------------------------------------------------------------------------
def test_norm_oracle_against_torch():
    g = np.random.default_rng(1)
    x, r, w = (synth.normal_bf16(g, s) for s in ((5, 256), (5, 256), (256,)))
    h, v = oracle.ref_rms_norm(x, r, w, 1e-5)
    tx, tr, tw = (torch.from_numpy(a.view(np.int16)).view(torch.bfloat16) for a in (x, r, w))
    th = tx + tr
    assert np.array_equal(h.view(np.int16), th.view(torch.int16).numpy())
    want = torch.nn.functional.rms_norm(th.double(), (256,), tw.double(), float(np.float32(1e-5)))
    assert np.allclose(v, want.numpy(), rtol=3 * 2.0 ** -24, atol=0)      # three roundings


def test_norm_codes_are_the_activation_quantizer_s():
    """On values that are bf16 already both quantize the same numbers: the same scales but for the last bit (a product
    here, a quotient there), the same codes where the scales are the same."""
    x = synth.normal_bf16(np.random.default_rng(2), (70, 256))
    v = oracle.decode_bf16(x).astype(np.float32)
    for fmt, want in (("int8", oracle.quantize_per_token(x, "int8")), ("fp8", oracle.quantize_per_token(x, "e4m3")),
                      ("block", oracle.quantize_fp8_block_act(x)), ("mxfp8", oracle.quantize_mxfp8_act(x)), ("mxfp4", oracle.quantize_mxfp4_act(x))):
        got = oracle.quantize_values(v, fmt)
        same = got[1].reshape(70, -1) == want[1].reshape(70, -1)
        assert np.allclose(got[1].astype(float), want[1].astype(float), rtol=2.0 ** -23, atol=0) and same.mean() > (0.2 if got[1].dtype == np.float32 else 0.999), fmt
        per = got[0].shape[1] // same.shape[1]
        assert np.array_equal(got[0].reshape(70, -1, per)[same], want[0].reshape(70, -1, per)[same]), fmt


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("is_value", [False, True])
def test_append_oracle_by_hand(fmt, is_value):
    """One page of four tokens, head size 2: a fresh scale, a growth by a power of two, a token that fits."""
    Q = 448.0 if fmt == "fp8" else 127.0
    pages, scales = np.full((2, 1, 2, 4) if is_value else (2, 1, 4, 2), 0xEE, np.uint8), np.full((2, 1), np.nan, np.float32)
    table = np.array([[1]], np.int32)

    def put(v, lens):
        x = synth.bf16_bits(np.array(v, np.float32)).reshape(-1, 1, 2)
        return oracle.ref_kv_append(fmt, x, is_value, np.array([0, len(x)], np.int32), [lens], table, *state)

    def held():
        c = state[0][1, 0].T if is_value else state[0][1, 0]
        c = c[:2]
        return (oracle.decode_int8(c.view(np.int8)) if fmt == "int8" else oracle.decode_e4m3(c)) * float(state[1][1, 0])
    state = (pages, scales)
    state = put([[1.0, -0.5]], 1)
    s = np.float32(1.0) / np.float32(Q)      # 1 * fp32(1 / Q)
    assert state[1][1, 0] == s and np.allclose(held()[0], [1.0, -0.5], rtol=0, atol=0.51 / Q if fmt == "int8" else 1e-7)
    assert np.isnan(state[1][0, 0]) and (state[0][0] == 0xEE).all()
    state = put([[3.0, 0.25]], 2)      # 3 / Q > s: twice that is too little, four times enough
    assert state[1][1, 0] == 4 * s
    assert np.allclose(held(), [[1.0, -0.5], [3.0, 0.25]], rtol=2.0 ** -4 if fmt == "fp8" else 0, atol=2.01 / Q)
    state = put([[4.0, 0.0]], 3)       # the largest that fits
    assert state[1][1, 0] == 4 * s
    c = state[0][1, 0].T if is_value else state[0][1, 0]
    assert (c[3] == 0xEE).all()        # the slot behind the end


def test_append_oracle_zeros_and_non_finite():
    x = np.array([[0, 0], [0x7F80, 0xFF80], [0x7FC0, 0x3F80]], np.uint16).reshape(3, 1, 2)     # zeros; inf, -inf; NaN, 1
    table, cu = np.array([[0]], np.int32), np.array([0, 1], np.int32)
    for fmt in ("fp8", "int8"):
        for is_value in (False, True):
            shape = (1, 1, 2, 16) if is_value else (1, 1, 16, 2)
            p, s = oracle.ref_kv_append(fmt, x[:1], is_value, cu, [1], table, np.full(shape, 0xEE, np.uint8), np.full((1, 1), 9, np.float32))
            assert s[0, 0] == 0
            p, s = oracle.ref_kv_append(fmt, x[2:], is_value, cu, [2], table, p, s)              # a page of zeros takes a new scale
            assert s[0, 0] == np.float32(1) / (448 if fmt == "fp8" else 127)
            c = (p[0, 0].T if is_value else p[0, 0])[:2]
            assert c[0].tolist() == [0, 0] and c[1].tolist() == [0x7F if fmt == "fp8" and not is_value else 0, 0x7E if fmt == "fp8" else 127]
            p, s = oracle.ref_kv_append(fmt, x[1:2], is_value, cu, [3], table, p, s)
            c = (p[0, 0].T if is_value else p[0, 0])[2]
            big = oracle.decode_bf16(np.array([0x7F7F], np.uint16))[0]
            v = (oracle.decode_e4m3(c) if fmt == "fp8" else oracle.decode_int8(c.view(np.int8))) * float(s[0, 0])
            assert np.allclose(v, [big, -big], rtol=2.0 ** -4) and np.isfinite(v).all()


def test_attention_oracle_against_torch():
    g = np.random.default_rng(3)
    for fmt in ("fp8", "int8"):
        c = kv_case(g, fmt, 2, 64, 16, [3, 1, 0, 5], [37, 1, 20, 5], behind=2)
        q = normal_rows(g, c["T"], 4, 64)
        keep = np.full(q.shape, 7.0)
        out, *_ = oracle.ref_attention(fmt, q, c["cu"], c["lens"], c["table"], c["k_pages"], c["v_pages"], c["k_scales"], c["v_scales"], 0.125, 0, keep)
        for b, n in enumerate(c["lens"]):
            first, new = c["cu"][b], c["cu"][b + 1] - c["cu"][b]
            if not new:
                continue
            pages = c["table"][b, :-(-n // 16)]
            val = oracle.decode_e4m3 if fmt == "fp8" else (lambda a: oracle.decode_int8(a.view(np.int8)))
            k = (val(c["k_pages"][pages]) * c["k_scales"][pages].astype(float)[:, :, None, None]).transpose(1, 0, 2, 3).reshape(2, -1, 64)[:, :n]
            v = (val(c["v_pages"][pages]) * c["v_scales"][pages].astype(float)[:, :, None, None]).transpose(1, 0, 3, 2).reshape(2, -1, 64)[:, :n]
            qq = torch.from_numpy(oracle.decode_bf16(q[first:first + new])).transpose(0, 1)
            mask = torch.tril(torch.ones(n, n, dtype=torch.bool))[n - new:]
            want = torch.nn.functional.scaled_dot_product_attention(qq, torch.from_numpy(k).repeat_interleave(2, 0), torch.from_numpy(v).repeat_interleave(2, 0),
                                                                    attn_mask=mask, scale=0.125)
            assert np.allclose(out[first:first + new], want.transpose(0, 1).numpy(), rtol=1e-10, atol=1e-12)
        assert (out[-2:] == 7.0).all()


def test_attention_oracle_empty_rows_and_left_out():
    g = np.random.default_rng(4)
    c = kv_case(g, "fp8", 1, 64, 16, [4, 2, 2], [2, 20, 40])
    q = normal_rows(g, c["T"], 1, 64)
    a = lambda **k: oracle.ref_attention("fp8", q, c["cu"], k.get("lens", c["lens"]), k.get("table", c["table"]), c["k_pages"], c["v_pages"],  # noqa: E731
                                         c["k_scales"], c["v_scales"], 0.1, k.get("window", 0), np.full(q.shape, 7.0), k.get("max_q"))[0]
    out = a()
    assert (out[:2] == 0).all() and (out[2:] != 0).all()       # positions -2 and -1 see nothing
    lost = c["table"].copy()
    lost[1] = -1
    assert (a(table=lost)[4:6] == 0).all()                     # no page left
    assert (a(max_q=3)[:4] == 7).all() and (a(max_q=3)[4:] != 7).all()
    assert (a(lens=[2, -1, 10000])[4:] == 7).all()
    # a window of one sees the token itself
    one = a(window=1)
    v = oracle.decode_e4m3(c["v_pages"][c["table"][1, 1], 0, :, 3]) * float(c["v_scales"][c["table"][1, 1], 0])
    assert np.allclose(one[5, 0], v)


def test_page_quotients_are_the_ieee_ones():
    """The append's quotient, a product with fp32(1 / s) and one correction, for every mantissa of a bf16 value and of a page's scale:
    the IEEE quotient (the fused operations in float64, where product and remainder are exact)."""
    m = (np.arange(128, 256) / 128).astype(np.float32)
    for unit in (np.float32(1) / np.float32(127), np.float32(1) / np.float32(448)):
        for s in m * unit:
            rs = np.float32(1) / s
            q = m * rs
            r = (m.astype(np.float64) - q.astype(np.float64) * np.float64(s)).astype(np.float32)
            got = (q.astype(np.float64) + r.astype(np.float64) * np.float64(rs)).astype(np.float32)
            assert np.array_equal(got, m / s)
    # and the product alone is not always
    assert any(not np.array_equal(m * (np.float32(1) / s), m / s) for s in m * (np.float32(1) / np.float32(127)))


# ---- what the bounds can see ------------------------------------------------------------------
@pytest.mark.parametrize("tokens", [40, 1000])
def test_bounds_see_mistakes(tokens):
    """An exact result rounded once passes both bounds; a lost last token, a token too many, a wrong head and a wrong page scale
    break the expected size."""
    g = np.random.default_rng(5)
    c = kv_case(g, "int8", 2, 64, 16, [4], [tokens])
    q = normal_rows(g, 4, 8, 64)
    run = lambda lens=tokens, **k: oracle.ref_attention("int8", k.get("q", q), c["cu"], [lens], c["table"], c["k_pages"], c["v_pages"],  # noqa: E731
                                                        k.get("ks", c["k_scales"]), k.get("vs", c["v_scales"]), 0.125, k.get("window", 0), np.zeros(q.shape))
    ref, size, spread, grain, reach = run()
    hard, var = attention_bounds(ref, size, spread, grain, reach, 64, tokens)
    rms = lambda got: float(np.sqrt(((got - ref) ** 2).sum() / var.sum()))  # noqa: E731
    rounded = oracle.decode_bf16(oracle.round_to_bf16(ref))
    assert (np.abs(rounded - ref) <= hard).all() and rms(rounded) < 1.0
    vs = c["v_scales"].copy()
    vs[c["table"][0, 1]] *= 1.5
    ks = c["k_scales"].copy()
    ks[c["table"][0, 1], 0] *= 1.5
    for wrong in (run(tokens - 1)[0], run(window=tokens - 2)[0], run(vs=vs)[0], run(ks=ks)[0], run(q=np.roll(q, 1, 1))[0]):
        assert rms(wrong) > 2.0


# ---- refusals ---------------------------------------------------------------------------------
@pytest.mark.parametrize("change,status", [
    (dict(fmt=6), INV), (dict(fmt=-1), INV), (dict(M=-1), INV), (dict(K=0), INV), (dict(K=12), UNS), (dict(K=65544), UNS), (dict(K=1 << 31), INV),
    (dict(fmt=NORM["mxfp8"], K=40), UNS), (dict(fmt=NORM["mxfp4"], K=16), UNS), (dict(fmt=NORM["block"], K=96), UNS),
    (dict(eps=0.0), INV), (dict(eps=-1e-6), INV), (dict(eps=math.nan), INV), (dict(eps=math.inf), INV), (dict(M=1 << 30, K=65536), UNS),
    (dict(r=None), INV), (dict(ro=None), INV), (dict(x=None), INV), (dict(y=None), INV), (dict(s=None), INV),
    (dict(x=8), INV), (dict(r=24), INV), (dict(w=8), INV), (dict(ro=24), INV), (dict(y=8), INV), (dict(s=18), INV), (dict(copy=8), INV),
    (dict(fmt=NORM["bf16"]), INV), (dict(fmt=NORM["bf16"], s=None, copy=64), INV),
    (dict(y=16), INV), (dict(y=32), INV), (dict(y=48), INV), (dict(copy=32), INV), (dict(copy=48), INV), (dict(copy=64), INV),
    (dict(ro=16, copy=16), INV), (dict(fmt=NORM["bf16"], s=None, ro=16, y=16), INV),
])
def test_norm_refusals(change, status):
    a = dict(fmt=NORM["fp8"], M=2, K=256, x=16, r=32, w=128, eps=1e-6, ro=48, y=64, s=96, copy=None) | change
    assert _status(hq.hq_rms_norm, a["fmt"], a["M"], a["K"], a["x"], a["r"], a["w"], a["eps"], a["ro"], a["y"], a["s"], a["copy"], stream=0) == status


KV = dict(fmt=0, H=8, D=128, P=16, pages=100, size=None)


def _desc(a):
    d = hq.make_kv_desc(a["fmt"], a["H"], a["D"], a["P"], a["pages"])
    if a["size"] is not None:
        d.struct_size = a["size"]
    return d


DESCS = [(dict(fmt=2), INV), (dict(fmt=-1), INV), (dict(H=0), INV), (dict(H=1025), INV), (dict(D=80), UNS), (dict(D=0), UNS), (dict(D=512), UNS),
         (dict(P=8), UNS), (dict(P=48), UNS), (dict(P=512), UNS), (dict(P=0), UNS), (dict(pages=0), INV), (dict(pages=-1), INV), (dict(size=20), INV)]
ARRAYS = [(dict(cu=None), INV), (dict(lens=None), INV), (dict(table=None), INV), (dict(kp=None), INV), (dict(vp=None), INV), (dict(ks=None), INV),
          (dict(vs=None), INV), (dict(cu=18), INV), (dict(lens=18), INV), (dict(table=18), INV), (dict(kp=8), INV), (dict(vp=8), INV), (dict(ks=18), INV),
          (dict(vs=18), INV), (dict(width=0), INV), (dict(width=-1), INV), (dict(width=(1 << 26) + 1), INV)]
SEQUENCES = [(dict(B=-1), INV), (dict(B=65536), INV), (dict(T=-1), INV), (dict(T=(1 << 24) + 1), INV), (dict(most=-1), INV), (dict(most=(1 << 24) + 1), INV)]


@pytest.mark.parametrize("change,status", DESCS + ARRAYS + SEQUENCES + [
    (dict(stride=1016), INV), (dict(stride=1028), INV), (dict(stride=(1 << 30) + 8), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(k=8), INV), (dict(v=8), INV),
    (dict(B=65535, T=1 << 24, most=1 << 12), UNS),
])
def test_append_refusals(change, status):
    a = dict(KV, B=4, T=10, most=5, k=16, v=16, stride=1024, cu=16, lens=16, table=16, width=9, kp=16, vp=16, ks=16, vs=16) | change
    assert _status(hq.hq_kv_append, _desc(a), a["B"], a["T"], a["most"], a["k"], a["v"], a["stride"], a["cu"], a["lens"], a["table"], a["width"], a["kp"],
                   a["vp"], a["ks"], a["vs"], stream=0) == status


@pytest.mark.parametrize("change,status", DESCS + ARRAYS + SEQUENCES + [
    (dict(Hq=0), INV), (dict(Hq=12), INV), (dict(Hq=1032), INV), (dict(max_kv=-1), INV), (dict(max_kv=(1 << 30) + 1), INV), (dict(stride=2040), INV),
    (dict(stride=2052), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(scale=-3e38), INV), (dict(window=-1), INV), (dict(q=None), INV), (dict(out=None), INV),
    (dict(q=8), INV), (dict(out=8), INV), (dict(ws=8), INV), (dict(ws=None), WSP), (dict(short=1), WSP), (dict(B=65535, T=1 << 24, most=1 << 24), UNS),
    (dict(q=48, out=48, stride=4096), INV),
])
def test_attention_refusals(change, status):
    a = dict(KV, B=4, T=10, most=5, Hq=16, max_kv=140000, q=16, stride=2048, cu=16, lens=16, table=16, width=9000, kp=16, vp=16, ks=16, vs=16, scale=0.1,
             window=0, out=48, ws=16, short=0) | change
    need = hq.hq_attention_workspace_bytes(_desc(KV), 4, 10, 16, 5, 140000)
    assert need > 0
    assert _status(hq.hq_attention, _desc(a), a["B"], a["T"], a["Hq"], a["most"], a["max_kv"], a["q"], a["stride"], a["cu"], a["lens"], a["table"], a["width"],
                   a["kp"], a["vp"], a["ks"], a["vs"], a["scale"], a["window"], a["out"], a["ws"], need - a["short"], stream=0) == status


def test_nothing_to_do():
    d = _desc(KV)
    hq.hq_rms_norm(NORM["fp8"], 0, 256, None, None, None, 1e-6, None, None, stream=0)
    for B, T, most in ((0, 10, 5), (4, 0, 5), (4, 10, 0)):
        hq.hq_kv_append(d, B, T, most, None, None, 1024, None, None, None, 0, None, None, None, None, stream=0)
        assert hq.hq_attention_workspace_bytes(d, B, T, 16, most, 1000) == 0
        hq.hq_attention(d, B, T, 16, most, 1000, None, 2048, None, None, None, 0, None, None, None, None, 0.1, 0, None, stream=0)


def test_sizes():
    for fmt in (0, 1):
        assert hq.hq_kv_cache_bytes(hq.make_kv_desc(fmt, 8, 96, 32, 7)) == 7 * 8 * 96 * 32
        assert hq.hq_kv_cache_bytes(hq.make_kv_desc(fmt, 1024, 256, 256, 1 << 20)) == 1 << 46        # past 32 bits
    assert hq.hq_kv_cache_bytes(hq.make_kv_desc(0, 8, 80, 32, 7)) == 0
    need = hq.hq_attention_workspace_bytes
    d = _desc(KV)
    assert need(d, 1, 1, 16, 1, 200000) > need(d, 1, 1, 16, 1, 2000) > 0 == need(d, 1, 1, 16, 1, 64)
    assert need(d, 1, 1, 12, 1, 2000) == 0                                                          # refused
    # room for rows, not for sequences times the longest: a prompt among single tokens
    assert need(d, 8, 40, 16, 33, 4096) <= need(d, 8, 8 * 33, 16, 33, 4096)


def test_workspace_grows_with_the_context():
    """A window shortens what a call plans for, as a smaller max_kv does; its workspace is sized without the window."""
    g = np.random.default_rng(21)
    shapes = [(43, 1, 1, 300, 300), (64, 2, 1, 129, 129), (5, 8, 3, 700, 300), (86, 1, 1, 300, 257)]
    shapes += [(int(g.integers(1, 90)), int(2 ** g.integers(0, 5)), int(g.integers(1, 6)), int(g.integers(1, 4000)), int(g.integers(1, 2000))) for _ in range(300)]
    for H, G, B, T, most in shapes:
        for D in (64, 128, 256):
            d = hq.make_kv_desc(0, H, D, 64, 100)
            last = 0
            for max_kv in sorted((0, 64, 65, 500, 1000, 1344, 2047, 2048, 2500, 4096, 5000, 2 * most - 1, 2 * most, 20000, 100000, 1 << 20)):
                n = hq.hq_attention_workspace_bytes(d, B, T, H * G, most, max_kv)
                assert n >= last, (H, G, B, T, most, D, max_kv)
                last = n


def test_norm_buffers_are_checked():
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    a = dict(fmt=NORM["fp8"], x=16, r=32, w=128, ro=48, y=64, s=96, copy=None)
    for change, what in ((dict(x=b(1, 256)), "x holds 512 bytes"), (dict(x=f(2, 256)), "x has elements"), (dict(r=b(256, 2).T), "residual must be contiguous"),
                         (dict(w=b(255)), "weight holds"), (dict(w=f(256)), "weight has elements"), (dict(ro=b(1, 256)), "residual_out holds"), (dict(y=u(511)), "y holds"),
                         (dict(y=b(512)), "y has elements"), (dict(s=f(1)), "y_scale holds"), (dict(s=u(8)), "y_scale has elements"), (dict(copy=b(2, 255)), "y_bf16 holds"),
                         (dict(fmt=NORM["mxfp8"], s=u(15)), "y_scale holds 15 bytes, 16"), (dict(fmt=NORM["mxfp4"], y=u(255)), "y holds 255 bytes, 256"),
                         (dict(fmt=NORM["block"], s=f(3)), "y_scale holds"), (dict(x=np.zeros((2, 256), np.uint16)), "x is a host array"),
                         (dict(x=b(2, 256)), "x must be on the current device")):
        c = a | change
        with pytest.raises(hq.HQError, match=what) as ei:
            hq.hq_rms_norm(c["fmt"], 2, 256, c["x"], c["r"], c["w"], 1e-6, c["ro"], c["y"], c["s"], c["copy"], stream=0)
        assert ei.value.status == INV


def test_cache_buffers_are_checked():
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    d = hq.make_kv_desc(0, 2, 64, 16, 3)
    a = dict(k=16, v=16, stride=128, cu=16, lens=16, table=16, kp=16, vp=16, ks=16, vs=16)
    wide = b(5, 6, 64)
    for change, what in ((dict(k=b(4, 2, 64)), r"k holds \(4, 2, 64\), 5 rows"), (dict(v=b(5, 127)), "v holds"), (dict(k=b(5, 2, 64).float()), "k holds torch.float32"),
                         (dict(k=b(5, 64, 2).transpose(1, 2)), "k must be contiguous within a row"), (dict(k=wide[:, 2:4]), "k has rows 384 elements apart, not 128"),
                         (dict(v=b(640)), "v holds"), (dict(cu=i(2)), "cu holds"), (dict(lens=i(1)), "kv_lens holds"), (dict(table=i(2, 3)), "page_table holds"),
                         (dict(table=i(4, 2).T), "page_table must be contiguous"), (dict(cu=i(3).long()), "cu has elements of 8 bytes"),
                         (dict(kp=torch.zeros(6143, dtype=torch.uint8)), "k_pages holds"), (dict(vp=torch.zeros(6143, dtype=torch.uint8)), "v_pages holds"),
                         (dict(ks=torch.zeros(5)), "k_scales holds"), (dict(vs=torch.zeros(6, dtype=torch.int32)), "v_scales holds torch.int32"),
                         (dict(stride=384, k=wide[:, 2:4]), "k must be on the current device"), (dict(k=b(5, 128)), "k must be on the current device")):
        c = a | change
        with pytest.raises(hq.HQError, match=what) as ei:
            hq.hq_kv_append(d, 2, 5, 4, c["k"], c["v"], c["stride"], c["cu"], c["lens"], c["table"], 4, c["kp"], c["vp"], c["ks"], c["vs"], stream=0)
        assert ei.value.status == INV
    a = dict(q=16, stride=256, out=48, ws=None) | {k: a[k] for k in ("cu", "lens", "table", "kp", "vp", "ks", "vs")}
    for change, what in ((dict(q=b(4, 4, 64)), "q holds"), (dict(q=wide[:, :4]), "q has rows 384"), (dict(out=b(5, 255)), "out holds"), (dict(out=b(5, 256).half()), "out holds torch.float16"),
                         (dict(ws=torch.zeros(8)), "ws holds"), (dict(kp=torch.zeros(6143, dtype=torch.uint8)), "k_pages holds"), (dict(q=b(5, 4, 64)), "q must be on")):
        c = a | change
        with pytest.raises(hq.HQError, match=what) as ei:
            hq.hq_attention(d, 2, 5, 4, 4, 64, c["q"], c["stride"], c["cu"], c["lens"], c["table"], 4, c["kp"], c["vp"], c["ks"], c["vs"], 0.1, 0, c["out"], c["ws"],
                            64 if c["ws"] is not None else 0, stream=0)
        assert ei.value.status == INV


def test_stream_of_another_device():
    class Stream:
        cuda_stream, device_index = 0, 1
    d = _desc(KV)
    for call in (lambda st: hq.hq_rms_norm(NORM["fp8"], 2, 256, 16, None, None, 1e-6, None, 64, 96, stream=st),
                 lambda st: hq.hq_kv_append(d, 1, 1, 1, 16, 16, 1024, 16, 16, 16, 1, 16, 16, 16, 16, stream=st),
                 lambda st: hq.hq_attention(d, 1, 1, 8, 1, 16, 16, 1024, 16, 16, 16, 1, 16, 16, 16, 16, 0.1, 0, 48, stream=st)):
        with pytest.raises(hq.HQError, match="stream must be on the current device"):
            call(Stream())


def test_page_quotients_at_any_scale():
    """The same quotient for scales of any mantissa, as pages hold that were filled elsewhere. The fused last step in float64: the sum of two exact
    terms, rounded there, decides the fp32 rounding but where that left it half way between two fp32."""
    g = np.random.default_rng(31)
    v = (np.arange(128, 256) / 128).astype(np.float32)
    ends = np.concatenate([np.arange(512), (1 << 23) - 1 - np.arange(512), (1 << 22) - 256 + np.arange(512)])
    for bits in np.array_split(np.unique(np.concatenate([ends, g.integers(0, 1 << 23, 100000)])), 20):
        s = ((np.uint32(0x3F800000) | bits.astype(np.uint32)).view(np.float32))[:, None]
        rs = np.float32(1) / s
        q = v * rs
        r = (v.astype(np.float64) - q.astype(np.float64) * s.astype(np.float64)).astype(np.float32)     # (exact before it is rounded)
        step = r.astype(np.float64) * rs.astype(np.float64)                   # exact
        z = q.astype(np.float64) + step
        lost = step - (z - q.astype(np.float64))                              # exact: the sum's own rounding
        half = (z.view(np.uint64) & 0x1FFFFFFF) == 0x10000000
        z = np.where(half & (lost != 0), np.nextafter(z, np.where(lost > 0, np.inf, -np.inf)), z)
        assert np.array_equal(z.astype(np.float32), v / s)
