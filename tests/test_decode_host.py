"""CPU checks of the decode-step calls: oracle pins, the fine-group layout, and every refusal (made on
the host before any launch, so they run without a GPU)."""
import math

import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_prepacked_amd as hq
import synth

from decode_harness import FORMATS, dequant, group_product_bound, prepack_host, product_bound, random_weights, route_case

INV, UNS, WSP = hq.HQ_ERR_INVALID_ARGUMENT, hq.HQ_ERR_UNSUPPORTED, hq.HQ_ERR_WORKSPACE
G32 = hq.DESC_W4A16_SYM_G32


# ---- oracle pins ------------------------------------------------------------------------------
def test_route_oracle_against_torch():
    g = np.random.default_rng(1)
    l = route_case(g, 9, 24, False)
    t = torch.from_numpy(l).double()
    ids, w = oracle.ref_route(l, None, "softmax", 5, renormalize=False, scale=2.0)
    top = torch.softmax(t, 1).topk(5, 1)
    assert np.array_equal(ids, top.indices.numpy()) and np.allclose(w, 2.0 * top.values.numpy(), rtol=1e-14)
    ids, w = oracle.ref_route(l, None, "sigmoid", 5)
    top = torch.sigmoid(t).topk(5, 1)
    assert np.array_equal(ids, top.indices.numpy())
    assert np.allclose(w, (top.values / top.values.sum(1, keepdim=True)).numpy(), rtol=1e-14)


def test_route_oracle_by_hand():
    l = np.log(np.array([[1.0, 3.0, 2.0, 2.0], [1.0, 1.0, 1.0, 1.0]]))
    ids, w = oracle.ref_route(l, None, "softmax", 2, renormalize=False)
    assert ids.tolist() == [[1, 2], [0, 1]] and np.allclose(w, [[3 / 8, 2 / 8], [1 / 4, 1 / 4]])
    # groups {0,1} and {2,3}: sums of two 4/8 and 4/8 -> the lower group
    ids, _ = oracle.ref_route(l[:1], None, "softmax", 2, n_group=2, topk_group=1)
    assert ids.tolist() == [[1, 0]]
    # by the largest alone group 0 wins too; a bias on expert 3 turns it
    ids, w = oracle.ref_route(l[:1], np.array([0, 0, 0, 0.5], np.float32), "softmax", 2, n_group=2, topk_group=1, group_top=1)
    assert ids.tolist() == [[3, 2]] and np.allclose(w, [[0.5, 0.5]])
    off = np.array([[-math.inf, math.nan, 1.0, -math.inf]])
    ids, w = oracle.ref_route(off, None, "softmax", 3)
    assert ids.tolist() == [[2, -1, -1]] and w.tolist() == [[1.0, 0.0, 0.0]]


def test_moe_oracle_is_the_layer_chain():
    """Token by token, entry by entry."""
    g = np.random.default_rng(2)
    T, topk, E, H, I = 3, 2, 4, 128, 128
    gu = [random_weights(g, "int4_g128", 2 * I, H) for _ in range(E)]
    dn = [random_weights(g, "int4_g128", H, I) for _ in range(E)]
    x = synth.normal_bf16(g, (T, H))
    ids = np.array([[0, 3], [1, -1], [2, 2]], np.int32)
    w = g.random((T, topk)).astype(np.float32)
    got = oracle.ref_moe_decode(x, ids, w, lambda e: dequant(gu[e], "int4_g128"), lambda e: dequant(dn[e], "int4_g128"))
    xf = oracle.decode_bf16(x)
    for t in range(T):
        want = np.zeros(H)
        for j in range(topk):
            if ids[t, j] < 0:
                continue
            y = dequant(gu[ids[t, j]], "int4_g128") @ xf[t]
            a = y[:I] / (1 + np.exp(-y[:I])) * y[I:]
            want += float(w[t, j]) * (dequant(dn[ids[t, j]], "int4_g128") @ a)
        assert np.allclose(got[t], want, rtol=1e-9, atol=1e-12)
    assert np.allclose(oracle.ref_gemv(x, dequant(gu[0], "int4_g128"), False), xf @ dequant(gu[0], "int4_g128").T)


def test_int4_groups_oracle_matches_the_128_group_one():
    g = np.random.default_rng(3)
    for fmt in ("int4_g128", "uint4_g128"):
        w = random_weights(g, fmt, 16, 256)
        assert np.array_equal(dequant(w, fmt), oracle.dequant_wna16(w["wq"], w["scales"], w["zeros"], 128))
    w = random_weights(g, "uint4_g32", 16, 128)
    v = dequant(w, "uint4_g32")
    code = lambda n, k: (int(w["wq"][n, k // 2]) >> (4 * (k % 2))) & 15  # noqa: E731
    for n, k in ((0, 0), (3, 31), (3, 32), (15, 127)):
        s = oracle.decode_bf16(w["scales"][n, k // 32:k // 32 + 1])[0]
        assert v[n, k] == (code(n, k) - int(w["zeros"][n, k // 32])) * s


# ---- prepack ----------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", [f for f in FORMATS if f.endswith(("128", "mxfp4", "int8", "fp8"))])
def test_prepack_of_shared_formats_is_the_ordinary_one(fmt):
    desc = FORMATS[fmt][0]
    g = np.random.default_rng(4)
    w = [random_weights(g, fmt, 48, 256) for _ in range(2)]
    out = np.zeros(hq.hq_prepacked_bytes(desc, 2, 48, 256), np.uint8)
    z = None if w[0]["zeros"] is None else np.stack([e["zeros"] for e in w])
    hq.hq_prepack_weights(desc, 2, 48, 256, np.stack([e["wq"] for e in w]), np.stack([e["scales"] for e in w]), z, out)
    assert np.array_equal(prepack_host(desc, w, 48, 256), out)


@pytest.mark.parametrize("fmt", ["int4_g32", "uint4_g32", "int4_g64", "uint4_g64"])
@pytest.mark.parametrize("E,N,K", [(1, 16, 128), (3, 48, 384)])
def test_fine_layout_round_trip(fmt, E, N, K):
    """Codes, scales and zeros read back from the documented positions of the layout."""
    desc, G, asym = FORMATS[fmt]
    g = np.random.default_rng(5)
    ws = [random_weights(g, fmt, N, K) for _ in range(E)]
    packed = prepack_host(desc, ws, N, K).reshape(E, -1)
    units, per = K // 128, 128 // G
    meta = 16 * per * 2 + (16 * per // 2 if asym else 0)
    align = lambda v: (v + 255) // 256 * 256  # noqa: E731
    m0 = align(N // 16 * units * 1024)
    assert packed.shape[1] == m0 + align(N // 16 * units * meta)
    for e, w in enumerate(ws):
        codes = np.zeros((N, K), np.uint8)
        for nt in range(N // 16):
            for kt in range(units):
                unit = packed[e, (nt * units + kt) * 1024:][:1024].view(np.uint32).reshape(64, 4)
                for l in range(64):
                    for d in range(4):
                        for p in range(8):
                            k = 128 * kt + 32 * d + 8 * (l >> 4) + 2 * (p & 3) + (p >> 2)
                            codes[16 * nt + (l & 15), k] = (int(unit[l, d]) >> (4 * p)) & 15
                m = packed[e, m0 + (nt * units + kt) * meta:][:meta]
                s = m[:32 * per].view(np.uint16).reshape(16, per)
                assert np.array_equal(s, w["scales"][16 * nt:16 * nt + 16, kt * per:(kt + 1) * per])
                if asym:
                    z = m[32 * per:].reshape(16, per // 2)
                    z = np.stack([z & 15, z >> 4], -1).reshape(16, per)
                    assert np.array_equal(z, w["zeros"][16 * nt:16 * nt + 16, kt * per:(kt + 1) * per])
        want = oracle.unpack_nibbles(w["wq"])
        assert np.array_equal(codes, want if asym else want ^ 8)


# ---- refusals ---------------------------------------------------------------------------------
def _status(f, *a, **k):
    with pytest.raises(hq.HQError) as ei:
        f(*a, **k)
    return ei.value.status


def test_descriptions():
    ok = hq.hq_decode_prepacked_bytes
    for desc, *_ in FORMATS.values():
        assert ok(desc, 1, 256, 512) > 0
        assert ok(hq.with_flags(desc, hq.HQ_COMPUTE_BATCH_INVARIANT), 1, 256, 512) == 0
        assert ok(desc, 1, 250, 512) == ok(desc, 1, 256, 448) == ok(desc, 0, 256, 512) == ok(desc, 1, 0, 512) == 0
    mk = hq.make_desc
    for bad in (mk(hq.HQ_W_INT4_SYM, 16, hq.HQ_SCALE_BF16, 0, hq.HQ_ACT_BF16),
                mk(hq.HQ_W_INT4_SYM, 32, hq.HQ_SCALE_BF16, 1, hq.HQ_ACT_BF16),
                mk(hq.HQ_W_UINT4_ASYM, 32, hq.HQ_SCALE_BF16, 0, hq.HQ_ACT_BF16),
                mk(hq.HQ_W_INT4_SYM, 32, hq.HQ_SCALE_FP32, 0, hq.HQ_ACT_BF16),
                mk(hq.HQ_W_FP4_E2M1, 64, hq.HQ_SCALE_E8M0, 0, hq.HQ_ACT_BF16),
                hq.DESC_W2A16_ASYM, hq.DESC_W3A16_ASYM, hq.DESC_W8A8, hq.DESC_W8A8_I32, hq.DESC_W4A8_MXFP4,
                hq.DESC_W4A4_MXFP4, hq.DESC_W4A8_MXFP8, hq.DESC_W8A8_FP8_BLOCK):
        assert ok(bad, 1, 256, 512) == 0
        assert _status(hq.hq_gemv, bad, 0, 1, 256, 512, 16, 16, 16, stream=0) == UNS
        assert hq.hq_moe_decode_workspace_bytes(bad, 1, 8, 16, 256, 512) == 0
    # the other calls still refuse the fine groups
    assert hq.hq_prepacked_bytes(hq.DESC_W4A16_ASYM_G32, 1, 256, 512) == 0
    assert _status(hq.hq_gemm, hq.DESC_W4A16_ASYM_G32, 4, 256, 512, 16, None, 16, 16, stream=0) == UNS


def test_prepack_size_overflow():
    """More bytes than a size_t counts: no size, and nothing is written."""
    huge = (65536, 1 << 30, 1 << 30)
    for desc, *_ in FORMATS.values():
        assert hq.hq_decode_prepacked_bytes(desc, *huge) == 0
        z = np.zeros(1, np.uint8) if desc.has_zero_point else None
        assert _status(hq.hq_decode_prepack_weights, desc, *huge, np.zeros(1, np.uint8), np.zeros(1, np.uint16), z, np.zeros(1, np.uint8)) == UNS


def test_prepack_refusals():
    g = np.random.default_rng(6)
    w = random_weights(g, "uint4_g32", 32, 256)
    out = np.zeros(hq.hq_decode_prepacked_bytes(hq.DESC_W4A16_ASYM_G32, 1, 32, 256), np.uint8)
    a = (1, 32, 256, w["wq"], w["scales"])
    assert _status(hq.hq_decode_prepack_weights, hq.DESC_W4A16_ASYM_G32, *a, None, out) == INV
    assert _status(hq.hq_decode_prepack_weights, hq.DESC_W4A16_SYM_G32, *a, w["zeros"], out) == INV
    assert _status(hq.hq_decode_prepack_weights, hq.DESC_W4A16_ASYM_G32, *a, w["zeros"], out[:-1]) == WSP
    assert _status(hq.hq_decode_prepack_weights, hq.DESC_W4A16_ASYM_G32, 0, 32, 256, w["wq"], w["scales"], w["zeros"], out) == INV


@pytest.mark.parametrize("change,status", [
    (dict(op=2), INV), (dict(M=-1), INV), (dict(M=65537), INV), (dict(N=250), UNS), (dict(K=500), UNS), (dict(N=0), INV),
    (dict(op=1, N=272), UNS), (dict(K=(1 << 24) + 128), UNS), (dict(M=1024, N=1 << 22), UNS), (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV),
    (dict(x=8), INV), (dict(w=24), INV), (dict(y=8), INV), (dict(N=(1 << 24) + 16), UNS),
])
def test_gemv_refusals(change, status):
    a = dict(op=0, M=4, N=256, K=512, x=16, w=16, y=16) | change
    assert _status(hq.hq_gemv, G32, a["op"], a["M"], a["N"], a["K"], a["x"], a["w"], a["y"], stream=0) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INV), (dict(T=17), UNS), (dict(topk=0), INV), (dict(topk=65), INV), (dict(E=0), INV), (dict(E=513), INV),
    (dict(H=200), UNS), (dict(I=1 << 23, topk=64, T=16), UNS), (dict(I=64), UNS), (dict(I=0), INV), (dict(x=None), INV), (dict(ids=None), INV), (dict(gu=None), INV),
    (dict(dn=None), INV), (dict(out=None), INV), (dict(x=8), INV), (dict(gu=8), INV), (dict(dn=8), INV), (dict(out=8), INV),
    (dict(ids=18), INV), (dict(w=18), INV), (dict(ws=8), INV), (dict(ws=None), WSP), (dict(short=1), WSP),
])
def test_moe_decode_refusals(change, status):
    a = dict(T=4, topk=8, E=16, H=256, I=512, x=16, ids=16, w=16, gu=16, dn=16, out=16, ws=16, short=0) | change
    need = hq.hq_moe_decode_workspace_bytes(G32, 4, 8, 16, 256, 512)
    assert need >= 4 * 8 * 512 * 2
    assert _status(hq.hq_moe_decode, G32, a["T"], a["topk"], a["E"], a["H"], a["I"], a["x"], a["ids"], a["w"], a["gu"], a["dn"],
                   a["out"], a["ws"], need - a["short"], stream=0) == status


@pytest.mark.parametrize("change,status", [
    (dict(score=2), INV), (dict(fmt=2), INV), (dict(T=-1), INV), (dict(T=(1 << 24) + 1), INV), (dict(E=0), UNS), (dict(E=513), UNS),
    (dict(groups=0), INV), (dict(groups=65), INV), (dict(groups=3), INV), (dict(keep=0), INV), (dict(keep=5), INV),
    (dict(top=0), INV), (dict(top=3), INV), (dict(topk=0), INV), (dict(topk=65), INV), (dict(topk=33), INV),
    (dict(scale=math.inf), INV), (dict(scale=math.nan), INV), (dict(logits=None), INV), (dict(ids=None), INV),
    (dict(weights=None), INV), (dict(logits=8), INV), (dict(bias=18), INV), (dict(ids=18), INV), (dict(weights=18), INV),
])
def test_route_refusals(change, status):
    a = dict(score=0, T=2, E=64, topk=8, logits=16, fmt=0, bias=None, groups=4, keep=2, top=2, scale=1.0, ids=16, weights=16) | change
    assert _status(hq.hq_moe_route, a["score"], a["T"], a["E"], a["topk"], a["logits"], a["fmt"], a["bias"], a["groups"], a["keep"],
                   a["top"], True, a["scale"], a["ids"], a["weights"], stream=0) == status


def test_nothing_to_do():
    hq.hq_gemv(G32, 0, 0, 256, 512, None, None, None, stream=0)
    hq.hq_moe_decode(G32, 0, 8, 16, 256, 512, None, None, None, None, None, None, stream=0)
    hq.hq_moe_route(0, 0, 64, 8, None, 0, None, 1, 1, 2, True, 1.0, None, None, stream=0)
    assert hq.hq_moe_decode_workspace_bytes(G32, 0, 8, 16, 256, 512) == 0


def test_buffers_are_checked():
    """What only the binding can see: host tensors, views that are not contiguous, short buffers."""
    x = torch.zeros((4, 512), dtype=torch.bfloat16)
    assert _status(hq.hq_gemv, G32, 0, 4, 256, 512, x, 16, 16, stream=0) == INV                       # on the host
    assert _status(hq.hq_gemv, G32, 0, 4, 256, 512, x.T, 16, 16, stream=0) == INV                     # not contiguous
    assert _status(hq.hq_gemv, G32, 0, 5, 256, 512, x, 16, 16, stream=0) == INV                       # four rows, five asked
    assert _status(hq.hq_moe_route, 0, 4, 512, 8, x, 0, None, 1, 1, 2, True, 1.0, 16, 16, stream=0) == INV   # bf16 held, fp32 asked
    with pytest.raises(hq.HQError, match="topk_ids has elements of 8 bytes"):                         # torch's own index type
        hq.hq_moe_decode(G32, 1, 8, 16, 256, 512, 16, torch.zeros(8, dtype=torch.int64), None, 16, 16, 16, 16, 1 << 20, stream=0)
    with pytest.raises(hq.HQError, match="x has elements of 4 bytes"):
        hq.hq_gemv(G32, 0, 4, 256, 512, x.float(), 16, 16, stream=0)
    w = torch.zeros(hq.hq_decode_prepacked_bytes(G32, 1, 256, 512) - 1, dtype=torch.uint8)
    with pytest.raises(hq.HQError, match="w_packed holds"):
        hq.hq_gemv(G32, 0, 4, 256, 512, 16, w, 16, stream=0)
    with pytest.raises(hq.HQError, match="w_down holds"):
        hq.hq_moe_decode(G32, 1, 8, 16, 256, 512, 16, 16, None, 16, w, 16, 16, 1 << 20, stream=0)
    ws = torch.zeros(8, dtype=torch.uint8)
    assert _status(hq.hq_moe_decode, G32, 1, 8, 16, 256, 512, 16, 16, None, 16, 16, 16, ws, 1 << 20, stream=0) == INV


def test_types_of_the_same_size_are_refused():
    """fp16 for bf16 and int32 for fp32 have the right size and the wrong values."""
    h, i = torch.zeros((4, 512), dtype=torch.float16), torch.zeros((4, 512), dtype=torch.int32)
    for call, what in ((lambda: hq.hq_gemv(G32, 0, 4, 256, 512, h, 16, 16, stream=0), "x"),
                       (lambda: hq.hq_gemv(G32, 0, 4, 256, 512, 16, 16, h, stream=0), "y"),
                       (lambda: hq.hq_moe_route(0, 4, 512, 8, h, hq.HQ_LOGITS_BF16, None, 1, 1, 2, True, 1.0, 16, 16, stream=0), "logits"),
                       (lambda: hq.hq_moe_route(0, 4, 512, 8, i, hq.HQ_LOGITS_FP32, None, 1, 1, 2, True, 1.0, 16, 16, stream=0), "logits"),
                       (lambda: hq.hq_moe_route(0, 4, 512, 8, 16, 0, i, 1, 1, 2, True, 1.0, 16, 16, stream=0), "bias"),
                       (lambda: hq.hq_moe_route(0, 4, 512, 8, 16, 0, None, 1, 1, 2, True, 1.0, i.float(), 16, stream=0), "topk_ids"),
                       (lambda: hq.hq_moe_route(0, 4, 512, 8, 16, 0, None, 1, 1, 2, True, 1.0, 16, i, stream=0), "topk_weights"),
                       (lambda: hq.hq_moe_decode(G32, 1, 8, 16, 256, 512, h, 16, None, 16, 16, 16, 16, 1 << 20, stream=0), "x"),
                       (lambda: hq.hq_moe_decode(G32, 1, 8, 16, 256, 512, 16, i.float(), None, 16, 16, 16, 16, 1 << 20, stream=0), "topk_ids"),
                       (lambda: hq.hq_moe_decode(G32, 1, 8, 16, 256, 512, 16, 16, i, 16, 16, 16, 16, 1 << 20, stream=0), "topk_weights"),
                       (lambda: hq.hq_moe_decode(G32, 1, 8, 16, 256, 512, 16, 16, None, 16, 16, h, 16, 1 << 20, stream=0), "out")):
        with pytest.raises(hq.HQError, match=rf"{what} holds torch\.\w+, not torch\.") as ei:
            call()
        assert ei.value.status == INV
    # a host array is no device buffer, whatever it holds
    with pytest.raises(hq.HQError, match="x is a host array"):
        hq.hq_gemv(G32, 0, 4, 256, 512, np.zeros((4, 512), np.uint16), 16, 16, stream=0)


def test_raw_bits_and_addresses_pass():
    """bf16 as its raw bits, addresses, and anything with a data_ptr()."""
    class Buffer:
        def data_ptr(self):
            return 16
    for x in (torch.zeros((4, 512), dtype=torch.int16), torch.zeros((4, 512), dtype=torch.uint16), torch.zeros((4, 512), dtype=torch.bfloat16)):
        with pytest.raises(hq.HQError, match="x must be on the current device"):   # the last check: every other one passed
            hq.hq_gemv(G32, 0, 4, 256, 512, x, 16, 16, stream=0)
    for x in (16, Buffer()):
        assert _status(hq.hq_gemv, G32, 2, 4, 256, 512, x, x, x, stream=0) == INV   # reaches the C side: unknown op
        assert "unknown op" in hq.hq_last_error()


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_prepack_checks_its_arrays(fmt):
    """Arrays shorter than the sizes say would be read past their end, and scales of another type misread."""
    desc = FORMATS[fmt][0]
    E, N, K = 2, 32, 256
    g = np.random.default_rng(7)
    w = [random_weights(g, fmt, N, K) for _ in range(E)]
    wq, sc = (np.stack([e[k] for e in w]) for k in ("wq", "scales"))
    z = None if w[0]["zeros"] is None else np.stack([e["zeros"] for e in w])
    out = np.zeros(hq.hq_decode_prepacked_bytes(desc, E, N, K), np.uint8)
    pack = lambda wq=wq, sc=sc, z=z, out=out: hq.hq_decode_prepack_weights(desc, E, N, K, wq, sc, z, out)  # noqa: E731
    want = pack().copy()
    bad = {"wq": [dict(wq=wq[:1]), dict(wq=wq.ravel()[:-1]), dict(wq=wq.astype(np.int32))],
           "scales": [dict(sc=sc[:1]), dict(sc=sc.ravel()[:-1]), dict(sc=sc.astype(np.float64)), dict(sc=sc.astype(np.float16))],
           "zeros": [] if z is None else [dict(z=z[:1]), dict(z=z.ravel()[:-1]), dict(z=z.astype(np.int64))]}
    if sc.dtype != np.float32:
        bad["scales"].append(dict(sc=sc.astype(np.float32)))
    for what, calls in bad.items():
        for call in calls:
            with pytest.raises(hq.HQError, match=f"^hq status 1: {what} ") as ei:
                pack(**call)
            assert ei.value.status == INV
    # any memory order, a larger array, and tensors on the host: as before
    assert np.array_equal(pack(wq=np.asfortranarray(wq), out=np.zeros_like(out)), want)
    assert np.array_equal(pack(wq=np.concatenate([wq, wq]), sc=np.concatenate([sc, sc]), out=np.zeros_like(out)), want)
    t = torch.zeros(out.size, dtype=torch.uint8)
    pack(wq=torch.from_numpy(wq), out=t)
    assert np.array_equal(t.numpy(), want)


def test_prepack_writes_only_into_whole_arrays():
    """A strided view counts its own bytes, but the call would write through its start over what lies between;
    a read-only array is somebody's constant."""
    g = np.random.default_rng(8)
    w = random_weights(g, "int4_g32", 32, 256)
    n = hq.hq_decode_prepacked_bytes(G32, 1, 32, 256)
    whole = np.zeros(2 * n, np.uint8)
    frozen = np.zeros(n, np.uint8)
    frozen.flags.writeable = False
    for out in (whole[::2], frozen, torch.zeros(2 * n, dtype=torch.uint8)[::2]):
        with pytest.raises(hq.HQError, match="^hq status 1: out ") as ei:
            hq.hq_decode_prepack_weights(G32, 1, 32, 256, w["wq"], w["scales"], None, out)
        assert ei.value.status == INV
    assert not whole.any() and not frozen.any()
    assert hq.hq_decode_prepack_weights(G32, 1, 32, 256, w["wq"], w["scales"], None, whole[:n]).any()


def test_stream_of_another_device():
    """The buffers are checked to be on the current device; a stream of another one would run the kernels there."""
    class Stream:
        cuda_stream, device_index = 0, 1
    for call in (lambda st: hq.hq_gemv(G32, 0, 4, 256, 512, 16, 16, 16, stream=st),
                 lambda st: hq.hq_moe_route(0, 4, 512, 8, 16, 0, None, 1, 1, 2, True, 1.0, 16, 16, stream=st),
                 lambda st: hq.hq_moe_decode(G32, 1, 8, 16, 256, 512, 16, 16, None, 16, 16, 16, 16, 1 << 20, stream=st)):
        with pytest.raises(hq.HQError, match="stream must be on the current device") as ei:
            call(Stream())
        assert ei.value.status == INV


def test_too_many_tokens_is_told_what_takes_them():
    """The grouped GEMMs take no weights in groups of 32 or 64: that error may not send a caller there."""
    call = lambda desc: hq.hq_moe_decode(desc, 17, 8, 16, 256, 512, 16, 16, None, 16, 16, 16, 16, 1 << 20, stream=0)  # noqa: E731
    for fmt, (desc, group, _) in FORMATS.items():
        with pytest.raises(hq.HQError) as ei:
            call(desc)
        fine = fmt.endswith(("_g32", "_g64"))
        assert ei.value.status == UNS and ("grouped GEMMs" in str(ei.value)) == (not fine) and ("calls of up to 16" in str(ei.value)) == fine
        assert (hq.hq_prepacked_bytes(desc, 16, 256, 512) == 0) == fine      # what the grouped GEMMs' prepack says


@pytest.mark.parametrize("fmt,M,K", [("int4_g32", 3, 14336), ("uint4_g64", 1, 4096), ("uint4_g128", 13, 8192), ("uint4_g32", 16, 4096)])
def test_large_products_check_sees_lost_terms(fmt, M, K):
    """At the sizes of a model: a lost scale group breaks the elementwise bound, and a lost k the relative one
    (2e-3 of the norm), which an exact result rounded once keeps."""
    g = np.random.default_rng(9)
    group = FORMATS[fmt][1]
    w = random_weights(g, fmt, 208, K)
    x = synth.normal_bf16(g, (M, K))
    v = dequant(w, fmt)
    ref = oracle.ref_gemv(x, v, False)
    bound = group_product_bound(x, w, fmt)
    assert (bound <= product_bound(x, w, fmt) * (1 + 2.0 ** -6)).all()
    rms, allowed = np.sqrt((ref ** 2).mean()), bound + 2.0 ** -8 * (np.abs(ref) + bound) + 2.0 ** -134
    worst = lambda got: float((np.abs(got - ref) / allowed).max())  # noqa: E731
    rel = lambda got: float(np.linalg.norm(got - ref) / np.linalg.norm(ref))  # noqa: E731
    rounded = oracle.decode_bf16(oracle.round_to_bf16(ref))
    size = np.linalg.norm(oracle.decode_bf16(x), axis=0)     # of each k in x
    assert worst(rounded) <= 1.0 and rel(rounded) < 2e-3
    for k0 in (0, K // 2, K - group):
        lost = v.copy()
        lost[:, k0:k0 + group] = 0.0
        got = oracle.ref_gemv(x, lost, False)
        assert worst(got) > 1.0 and rel(got) > 2e-3, (k0, worst(got), rel(got), float(bound.mean() / rms))
        k = k0 + int(np.argmax(size[k0:k0 + group]))         # (one whose x is next to nothing no check could see)
        lost = v.copy()
        lost[:, k] = 0.0
        assert rel(oracle.ref_gemv(x, lost, False)) > 2e-3


def test_prepack_into_memory_of_one_s_own():
    """Anything with a data_ptr() and its bytes (a mapped file, an arena) is taken as it is."""
    g = np.random.default_rng(10)
    w = random_weights(g, "int4_g32", 32, 256)
    memory = np.zeros(hq.hq_decode_prepacked_bytes(G32, 1, 32, 256), np.uint8)

    class Arena:
        nbytes = memory.nbytes

        def data_ptr(self):
            return memory.ctypes.data
    hq.hq_decode_prepack_weights(G32, 1, 32, 256, w["wq"], w["scales"], None, Arena())
    assert np.array_equal(memory, prepack_host(G32, w, 32, 256))
