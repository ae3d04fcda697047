"""GPU parity of the RMS norm (residual's addition, norm, quantized or bf16 output) with the oracle: the stream, codes and
scales bit for bit, since both sides take every rounding in the same order."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_prepacked_amd as hq
import synth

from gpu_harness import BF16_NAN_BITS, DEV, say, to_dev
from layer_harness import NORM

pytestmark = pytest.mark.gpu

UNIT = {"block": 128, "mxfp8": 32, "mxfp4": 32}
PAD = 64


def _scale_count(fmt, M, K):
    return {"bf16": 0, "int8": M, "fp8": M}.get(fmt, M * K // UNIT.get(fmt, 1))


class Buffers:
    """Outputs with a pad behind each that has to stay."""

    def __init__(self, fmt, M, K, residual, both):
        n = M * K
        self.n, self.fmt = n, fmt
        self.codes = n * 2 if fmt == "bf16" else n // 2 if fmt == "mxfp4" else n
        self.scale_bytes = _scale_count(fmt, M, K) * (1 if fmt.startswith("mx") else 4)
        self.y = torch.full((self.codes + PAD,), 0xA5, dtype=torch.uint8, device=DEV)
        self.s = torch.full((self.scale_bytes + PAD,), 0xA5, dtype=torch.uint8, device=DEV) if fmt != "bf16" else None
        self.sum = torch.full((n + PAD,), BF16_NAN_BITS, dtype=torch.int16, device=DEV) if residual else None
        self.copy = torch.full((n + PAD,), BF16_NAN_BITS, dtype=torch.int16, device=DEV) if both else None

    def args(self):
        y = self.y.view(torch.int16) if self.fmt == "bf16" else self.y
        s = None if self.s is None else self.s if self.fmt.startswith("mx") else self.s.view(torch.float32)
        return self.sum, y, s, self.copy

    def untouched(self):
        assert bool((self.y[self.codes:] == 0xA5).all())
        assert self.s is None or bool((self.s[self.scale_bytes:] == 0xA5).all())
        for t in (self.sum, self.copy):
            assert t is None or bool((t[self.n:] == BF16_NAN_BITS).all())


def _run(fmt, x, r, w, eps=1e-6, both=False, stream=None):
    M, K = x.shape
    out = Buffers(fmt, M, K, r is not None, both)
    up = lambda a: None if a is None else to_dev(a)  # noqa: E731
    total, y, s, copy = out.args()
    hq.hq_rms_norm(NORM[fmt], M, K, up(x), up(r), up(w), eps, total, y, s, copy, stream=stream)
    torch.cuda.synchronize()
    out.untouched()
    return out


def _bits16(t, n):
    return t[:n].cpu().numpy().view(np.uint16)


def _check(fmt, x, r, w, eps=1e-6, both=False):
    M, K = x.shape
    out = _run(fmt, x, r, w, eps, both)
    h, v = oracle.ref_rms_norm(x, r, w, eps)
    if r is not None:
        assert np.array_equal(_bits16(out.sum, M * K).reshape(M, K), h), "residual_out"
    if both:
        assert np.array_equal(_bits16(out.copy, M * K).reshape(M, K), oracle.round_to_bf16(v)), "y_bf16"
    y = out.y[:out.codes].cpu().numpy()
    if fmt == "bf16":
        assert np.array_equal(y.view(np.uint16).reshape(M, K), oracle.round_to_bf16(v)), "y"
        return
    codes, scales = oracle.quantize_values(v, fmt)
    got = out.s[:out.scale_bytes].cpu().numpy().view(scales.dtype).reshape(scales.shape)
    assert np.array_equal(got, scales), "scales"
    bad = np.flatnonzero(y.view(np.uint8) != codes.ravel().view(np.uint8))
    assert bad.size == 0, f"{bad.size} codes differ, first at {bad[:5]}"


SIZES = [(1, 128), (1, 4096), (3, 512), (5, 640), (4, 1024), (7, 1152), (9, 2048), (2, 2176), (6, 4096), (3, 5120), (2, 7168), (3, 8192), (2, 8320), (2, 16384),
         (2, 16512), (1, 32768), (2, 33024), (1, 65536), (130, 256),
         (1024, 1152), (1027, 2048), (1025, 6144), (1024, 6272), (1023, 8192), (256, 2304), (257, 4096)]


@pytest.mark.parametrize("fmt", list(NORM))
@pytest.mark.parametrize("M,K", SIZES)
def test_norm_matches_oracle(fmt, M, K):
    """Every number of threads and chunks, on both sides of each border."""
    g = np.random.default_rng([M, K])
    if fmt == "mxfp4" and K > 8320:
        M = 1
    x, r = synth.normal_bf16(g, (M, K), 3.0), synth.normal_bf16(g, (M, K), 0.7)
    w = synth.bf16_bits(g.uniform(0.2, 2.0, K).astype(np.float32))
    say(f"[norm {fmt}] M={M} K={K}")
    _check(fmt, x, r, w, both=fmt != "bf16")
    _check(fmt, x, None, w)


@pytest.mark.parametrize("fmt", list(NORM))
@pytest.mark.parametrize("K", [8, 24, 32, 96, 136, 504, 520, 1032, 2056, 4104, 8200, 16392])
def test_norm_odd_widths(fmt, K):
    """K that fills no wave, and K that ends inside one."""
    if K % UNIT.get(fmt, 8):
        K = -(-K // UNIT[fmt]) * UNIT[fmt]
    g = np.random.default_rng(K)
    _check(fmt, synth.normal_bf16(g, (5, K), 20.0), synth.normal_bf16(g, (5, K)), None, eps=1e-5, both=fmt != "bf16")


@pytest.mark.parametrize("fmt", list(NORM))
def test_norm_edge_rows(fmt):
    """Rows of zeros (eps decides), of one value, of subnormals, of the largest values; a weight with zeros and negative values; sums that
    cancel; eps that outweighs the row."""
    K = 256
    g = np.random.default_rng(5)
    rows = [np.zeros(K), np.full(K, -3.0), np.linspace(-1, 1, K) * 1e-38, np.where(np.arange(K) % 2, 3.3e38, -3.3e38),
            np.where(np.arange(K) == 7, 1000.0, 1e-3), np.linspace(-2.0 ** -8, 2.0 ** -8, K), np.full(K, 2.0 ** -133), g.normal(0, 1e-12, K)]
    x = synth.bf16_bits(np.array(rows, np.float32))
    w = g.uniform(-2, 2, K).astype(np.float32)
    w[::5] = 0
    r = x.copy()
    r[4] ^= 0x8000                       # cancels
    for eps in (1e-6, 1e-12, 100.0):
        _check(fmt, x, None, synth.bf16_bits(w), eps=eps, both=fmt != "bf16")
        keep = [0, 1, 2, 4, 5, 6, 7]     # (3.3e38 twice is infinity)
        _check(fmt, x[keep], r[keep], synth.bf16_bits(w), eps=eps)


@pytest.mark.parametrize("fmt", list(NORM))
def test_norm_bad_rows_alone(fmt):
    """NaN and infinity in one row: the others as without it; bf16 results follow the formula."""
    g = np.random.default_rng(6)
    x = synth.normal_bf16(g, (6, 512))
    w = synth.normal_bf16(g, (512,))
    want = _run(fmt, x, None, w, both=fmt != "bf16")
    bad = x.copy()
    bad[1, 3], bad[4, 100] = 0x7FC0, 0xFF80
    got = _run(fmt, bad, None, w, both=fmt != "bf16")
    rows = [0, 2, 3, 5]
    per = want.codes // 6
    assert bool((got.y[:want.codes].view(6, per)[rows] == want.y[:want.codes].view(6, per)[rows]).all())
    if fmt != "bf16":
        per = want.scale_bytes // 6
        assert bool((got.s[:want.scale_bytes].view(6, per)[rows] == want.s[:want.scale_bytes].view(6, per)[rows]).all())
    copy = got.y[:got.codes].view(torch.bfloat16) if fmt == "bf16" else got.copy[:got.n].view(torch.bfloat16)
    copy = copy.view(6, 512).float()
    assert bool(torch.isnan(copy[1]).all())                                    # a NaN in the sum
    others = torch.arange(512, device=DEV) != 100
    assert bool(torch.isnan(copy[4, 100])) and bool((copy[4, others] == 0).all())   # 1 / sqrt(inf) = 0


def test_norm_scale_rule_of_every_quotient():
    """The codes go by the IEEE quotient: rows whose largest value sweeps over many exponents and mantissas, with values on
    both sides of every rounding border."""
    g = np.random.default_rng(7)
    K = 2048
    x = (g.uniform(-1, 1, (64, K)) * np.ldexp(g.uniform(1, 2, (64, 1)), np.arange(-32, 32)[:, None])).astype(np.float32)
    for fmt in ("int8", "fp8", "block"):
        _check(fmt, synth.bf16_bits(x), None, None, eps=1e-30)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8"])
def test_norm_in_place(fmt):
    """residual_out over the residual or over x; the bf16 result over x."""
    g = np.random.default_rng(8)
    x, r, w = synth.normal_bf16(g, (9, 4096)), synth.normal_bf16(g, (9, 4096)), synth.normal_bf16(g, (4096,))
    h, v = oracle.ref_rms_norm(x, r, w, 1e-6)
    for over in ("residual", "x"):
        dx, dr = to_dev(x), to_dev(r)
        total = dr if over == "residual" else dx
        out = Buffers(fmt, 9, 4096, False, False)
        _, y, s, _ = out.args()
        copy = None
        if over == "residual":
            if fmt == "bf16":
                y = dx
            else:
                copy = dx
        hq.hq_rms_norm(NORM[fmt], 9, 4096, dx, dr, to_dev(w), 1e-6, total, y, s, copy)
        torch.cuda.synchronize()
        assert np.array_equal(total.cpu().numpy().view(np.uint16), h)
        if over == "residual":
            assert np.array_equal(dx.cpu().numpy().view(np.uint16), oracle.round_to_bf16(v))
        if fmt == "fp8":
            assert np.array_equal(y[:9 * 4096].cpu().numpy().reshape(9, 4096), oracle.quantize_values(v, "fp8")[0])


def test_norm_many_rows():
    """More rows than one launch has workgroups for in a single pass of small widths, and rows of a prompt."""
    for M, K, fmt in ((4194304 + 9, 8, "int8"), (1048576 + 5, 1032, "fp8"), (4099, 5120, "mxfp8")):
        g = torch.Generator(device=DEV)
        g.manual_seed(M)
        x = torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16)
        y = torch.empty((M, K), dtype=torch.uint8, device=DEV)
        s = torch.empty((M, K // 32), dtype=torch.uint8, device=DEV) if fmt == "mxfp8" else torch.empty(M, device=DEV)
        hq.hq_rms_norm(NORM[fmt], M, K, x, None, None, 1e-6, None, y, s)
        torch.cuda.synchronize()
        rows = np.concatenate([np.arange(4), g_rows(M), np.arange(M - 4, M)])
        at = torch.from_numpy(rows).to(DEV)
        _, v = oracle.ref_rms_norm(x[at].view(torch.int16).cpu().numpy().view(np.uint16), None, None, 1e-6)
        codes, scales = oracle.quantize_values(v, fmt)
        assert np.array_equal(y[at].cpu().numpy(), codes.view(np.uint8)) and np.array_equal(s[at].cpu().numpy(), scales)


def g_rows(M):
    return np.random.default_rng(M).integers(0, M, 60)


def test_norm_is_the_quantizer_on_bf16_values():
    """With a weight of powers of two and rows whose norm is exactly one, the codes are hq_quantize_activations' own."""
    K = 256
    x = synth.bf16_bits(np.where(np.random.default_rng(9).random((8, K)) < 0.5, -1, 1).astype(np.float32))
    w = synth.bf16_bits(np.ldexp(1.0, np.random.default_rng(10).integers(-6, 6, K)).astype(np.float32))
    product = synth.bf16_bits(synth.bf16_bits_to_f32(x) * synth.bf16_bits_to_f32(w))
    for fmt in ("int8", "fp8", "block", "mxfp8", "mxfp4"):
        out = _run(fmt, x, None, w, eps=1e-30)
        q = torch.empty(out.codes, dtype=torch.uint8, device=DEV)
        s = torch.empty(out.scale_bytes, dtype=torch.uint8, device=DEV)
        hq.hq_quantize_activations(NORM[fmt], 8, K, to_dev(product), q, s)
        torch.cuda.synchronize()
        assert bool((q == out.y[:out.codes]).all()) and bool((s == out.s[:out.scale_bytes]).all()), fmt


def test_norm_graph_and_stream():
    """Captured and replayed with the program's own work between, and on another stream."""
    g = np.random.default_rng(11)
    M, K = 17, 4096
    x = to_dev(synth.normal_bf16(g, (M, K)))
    r = to_dev(synth.normal_bf16(g, (M, K)))
    w = to_dev(synth.normal_bf16(g, (K,)))
    y, s, total = torch.empty((M, K), dtype=torch.uint8, device=DEV), torch.empty(M, device=DEV), torch.empty_like(x)
    call = lambda stream=None: hq.hq_rms_norm(NORM["fp8"], M, K, x, r, w, 1e-6, total, y, s, stream=stream)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    side = torch.cuda.Stream()
    for k in range(4):
        x.copy_(to_dev(synth.normal_bf16(g, (M, K))))
        _, v = oracle.ref_rms_norm(x.cpu().numpy().view(np.uint16), r.cpu().numpy().view(np.uint16), w.cpu().numpy().view(np.uint16), 1e-6)
        codes, scales = oracle.quantize_values(v, "fp8")
        for how in ("graph", "stream"):
            y.fill_(0)
            s.fill_(0)
            if how == "graph":
                graph.replay()
            else:
                side.wait_stream(torch.cuda.current_stream())
                call(side)
                torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            assert np.array_equal(y.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), scales), how
