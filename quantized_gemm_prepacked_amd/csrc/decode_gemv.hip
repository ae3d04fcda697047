// decode_gemv.hip -- hq_gemv: y = x . W^T for one to a few rows, plain or gated (silu(gate) * up).
//
// Bound by the packed weights' bytes from some 20 MB on: 14336 x 4096 at M = 1 in groups of 64 reads 31.8 MB
// in 7.8 us (4.1 TB/s; a kernel that only reads that much takes 6.7), the gated 2 x 14336 x 4096 at M = 3 66 MB in
// 12.4 (5.3 TB/s; 11.4); below, by a launch's own time (2.5 us for 256 x 512, 2.2 back to back). With five rows or
// more the rows' copies into LDS count too, since every workgroup reads all of x: 8208 x 8192 at M = 13 takes 11.4
// us for 36.8 MB (3.2 TB/s), with 171 workgroups copying 256 KiB each beside them.
// A workgroup owns NT tiles of 16 output channels (gated: the gate and the up tile of the same
// outputs, in pairs) and one row block; its NW waves take every NW-th K unit each (decode_ops.h) and
// add their partial tiles through LDS, in wave order.
#include <hip/hip_runtime.h>

#include "decode_ops.h"
#include "elementwise_ops.h"
#include "internal.h"

namespace hq {

namespace {

struct GemvParams {
  DecW W;
  const uint16_t* x;
  uint16_t* y;
  int M, N, K;      // N: weight rows (gated: two outputs' worth)
};

template <int F, int AM, int NT, int NW, int D, bool GATED>
__global__ __launch_bounds__(NW * 64) void gemv_kernel(GemvParams p) {
  constexpr int E = dec_elems<AM>();
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = blockIdx.y * AM;
  const int out_tiles = p.N / 16 / (GATED ? 2 : 1);
  constexpr int OT = GATED ? NT / 2 : NT;     // output tiles of the workgroup
  const int ot0 = blockIdx.x * OT;

  // tile t of the wave: output tile ot0 + t (gated: t / 2, even t the gate, odd t the up tile); a group
  // past the last output tile repeats it and stores nothing of it
  DecTile<F> tiles[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int ot = min(ot0 + (GATED ? t / 2 : t), out_tiles - 1);
    tiles[t] = dec_tile<F>(p.W, p.W.w, GATED && (t & 1) ? ot + out_tiles : ot);
  }
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int n = p.W.units > wave ? (p.W.units - wave + NW - 1) / NW : 0;
  dec_stream<F, AM, NT, D>(
      n, dec_rsrc(p.x + size_t(row0) * p.K, uint32_t(min(AM, p.M - row0)) * p.K * 2), smem + wave * dec_wave_lds<AM, D>(), lane, acc, [](int) __attribute__((always_inline)) {},
      [&](int t) __attribute__((always_inline)) { return tiles[t]; },
      [&](int i, int) __attribute__((always_inline)) { return wave + i * NW; },
      [&](int i, int r) __attribute__((always_inline)) {
        return uint32_t(min(r, p.M - 1 - row0)) * (p.K * 2) + uint32_t(wave + i * NW) * 256;
      },
      [](int, const DecUnit<F>(&)[NT]) __attribute__((always_inline)) {});

  float(*red)[NT][E][64] = reinterpret_cast<float(*)[NT][E][64]>(smem);
  __syncthreads();   // every wave is done with its activations
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < E; ++i) red[wave][t][i][lane] = dec_value<F, AM>(acc[t], i);
  __syncthreads();
  for (int q = threadIdx.x; q < OT * E * 64; q += NW * 64) {
    const int le = q & 63, i = (q >> 6) % E, o = (q >> 6) / E;
    const int r = AM == 16 ? 4 * (le >> 4) + i : le >> 4;
    const int ot = ot0 + o;
    if (ot >= out_tiles || r >= AM || row0 + r >= p.M) continue;
    const int n = ot * 16 + (le & 15);
    const int t = GATED ? 2 * o : o;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w][t][i][le];
    if constexpr (DecTraits<F>::kW8) v *= reinterpret_cast<const float*>(p.W.w + p.W.scales_off)[n];
    if constexpr (GATED) {
      float u = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) u += red[w][t + 1][i][le];
      if constexpr (DecTraits<F>::kW8) u *= reinterpret_cast<const float*>(p.W.w + p.W.scales_off)[n + p.N / 2];
      v = silu(v) * u;
    }
    p.y[size_t(row0 + r) * (out_tiles * 16) + n] = f32_to_bf16_rne(v);
  }
}

template <int F, int AM, int NT, int NW, int D, bool GATED>
hipError_t launch_one(const GemvParams& p, hipStream_t s) {
  constexpr int red = NW * NT * dec_elems<AM>() * 256, rows = NW * dec_wave_lds<AM, D>();
  constexpr int lds = red > rows ? red : rows;
  static_assert(lds <= 160 * 1024, "LDS");
  static_assert(!GATED || NT % 2 == 0, "gate and up tiles come in pairs: with none a workgroup, the grid below would divide by zero");
  auto kern = gemv_kernel<F, AM, NT, NW, D, GATED>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  constexpr int OT = GATED ? NT / 2 : NT;
  const int out_tiles = p.N / 16 / (GATED ? 2 : 1);
  hipLaunchKernelGGL(kern, dim3(unsigned((out_tiles + OT - 1) / OT), unsigned((p.M + AM - 1) / AM)), dim3(NW * 64), lds, s, p);
  return hipGetLastError();
}

// Tile groups (of lo .. hi tiles) per workgroup: what leaves the fullest CU the fewest tiles when the
// workgroups are dealt over the 256 CUs, ties to the more (or fewer) tiles.
int tiles_per_workgroup(int tiles, int lo, int hi, bool ties_to_more) {
  int best = lo, cost = 1 << 30;
  for (int nt = lo; nt <= hi; ++nt) {
    const int c = ((tiles + nt - 1) / nt + 255) / 256 * nt;
    if (c < cost || (c == cost && ties_to_more)) {
      best = nt;
      cost = c;
    }
  }
  return best;
}

// Tiles per workgroup (NT), waves and ring depth, measured on one WNA16 group-128 layer a launch, weights
// from HBM, us (NT x waves x D):
//   up to 256 output tiles: one a workgroup, so every CU has one, and a deep ring (M = 1: 4096 x 14336 8.0 as
//   1x8x4, 11.5 as 2x8x2, 15.2 as 4x8x2; 2048 x 8192 4.7, 6.2, 9.3); with two K units a wave or less a
//   ring of two (as 1x8x2 / 1x8x4: 2048 x 2048 2.87 / 3.16, 2048 x 2560 3.24 / 3.16; groups of 32 alike)
//   more: two to four tiles share the activations' reads and row sums (M = 1: 14336 x 4096 7.5 as 2x8x2,
//   8.5 as 1x8x4; M = 16: 28672 x 8192 26 as 4x8x2, 31 as 2x8x2, 48 as 1x8x3), as many as fill the CUs
//   evenly (M = 16: 8192 x 8192 11.0 as 2x8x2, 13.7 as 4x8x2; one tile more, 8208 x 8192, 15.4 as 2x8x2,
//   12.5 as 3x8x2, 13.9 as 4x8x2). Groups of 32 too, whose four tiles need the most registers (135 of them;
//   12320 x 4096, M = 16: 9.6 as 4x8x2, 10.5 as 3x8x2)
//   gated: pairs of a gate and an up tile; more waves where K is long and pairs are few (M = 1, as 2x16x2 / 2x8x2:
//   64 pairs x 8192 6.1 / 6.4, x 6144 5.6 / 5.4; the other end, 255 pairs x 8192, is 8.5 / 8.4, and groups of 32
//   gain nothing: 64 pairs x 8192 6.9 / 6.9)
template <int F, bool GATED>
hipError_t launch_rows(const GemvParams& p, hipStream_t s) {
  const int tiles = p.N / 16 / (GATED ? 2 : 1);
  if constexpr (GATED) {
    if (p.M == 1) return tiles < 256 && p.W.units >= 64 ? launch_one<F, 1, 2, 16, 2, true>(p, s) : launch_one<F, 1, 2, 8, 2, true>(p, s);
    if (p.M <= 4) return launch_one<F, 4, 2, 8, 2, true>(p, s);
    return tiles_per_workgroup(tiles, 1, 2, true) == 1 ? launch_one<F, 16, 2, 8, 2, true>(p, s) : launch_one<F, 16, 4, 8, 2, true>(p, s);
  } else {
    if (p.M == 1) {
      if (tiles <= 256) return p.W.units <= 16 ? launch_one<F, 1, 1, 8, 2, false>(p, s) : launch_one<F, 1, 1, 8, 4, false>(p, s);
      return tiles_per_workgroup(tiles, 2, 3, false) == 2 ? launch_one<F, 1, 2, 8, 2, false>(p, s) : launch_one<F, 1, 3, 8, 2, false>(p, s);
    }
    if (p.M <= 4) {
      if (tiles <= 256) return launch_one<F, 4, 1, 8, 3, false>(p, s);
      return tiles_per_workgroup(tiles, 2, 3, false) == 2 ? launch_one<F, 4, 2, 8, 2, false>(p, s) : launch_one<F, 4, 3, 8, 2, false>(p, s);
    }
    if (tiles <= 256) return launch_one<F, 16, 1, 8, 3, false>(p, s);
    switch (tiles_per_workgroup(tiles, 2, 4, true)) {
      case 2: return launch_one<F, 16, 2, 8, 2, false>(p, s);
      case 3: return launch_one<F, 16, 3, 8, 2, false>(p, s);
      default: return launch_one<F, 16, 4, 8, 2, false>(p, s);
    }
  }
}

}  // namespace

DecW dec_weights(const Combo& c, const uint8_t* w, int64_t N, int64_t K) {
  const PackedLayout L = c.fine_group ? make_fine_layout(c.fine_group, c.asym, N, K) : make_layout(c.fam, c.asym, N, K);
  return DecW{w, L.scales_off, L.zeros_off, L.expert_stride, int(K / 128)};
}

int dec_format(const Combo& c) {
  if (c.fam == FAM_WNA16) return (c.fine_group == 32 ? DF_G32 : c.fine_group == 64 ? DF_G64 : DF_G128) + (c.asym ? 1 : 0);
  return c.fam == FAM_MXW4A16 ? DF_MXFP4 : c.fam == FAM_W8A16 ? DF_INT8 : DF_FP8;
}

template <int F>
static hipError_t gemv_fmt(const GemvCall& g, hipStream_t s) {
  const GemvParams p{dec_weights(g.c, g.w, g.N, g.K), static_cast<const uint16_t*>(g.x), static_cast<uint16_t*>(g.y),
                     int(g.M), int(g.N), int(g.K)};
  return g.gated ? launch_rows<F, true>(p, s) : launch_rows<F, false>(p, s);
}

hipError_t launch_gemv(const GemvCall& g, hipStream_t s) {
  switch (dec_format(g.c)) {
    case DF_G128: return gemv_fmt<DF_G128>(g, s);
    case DF_G128Z: return gemv_fmt<DF_G128Z>(g, s);
    case DF_G64: return gemv_fmt<DF_G64>(g, s);
    case DF_G64Z: return gemv_fmt<DF_G64Z>(g, s);
    case DF_G32: return gemv_fmt<DF_G32>(g, s);
    case DF_G32Z: return gemv_fmt<DF_G32Z>(g, s);
    case DF_MXFP4: return gemv_fmt<DF_MXFP4>(g, s);
    case DF_INT8: return gemv_fmt<DF_INT8>(g, s);
    default: return gemv_fmt<DF_FP8>(g, s);
  }
}

}  // namespace hq
