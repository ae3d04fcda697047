// decode.hip -- the decode step's matrix-vector kernels: y = x . W^T for one to a few rows (plain, or
// gated: silu(gate) * up), and the MoE layer for a few tokens in two launches.
//
// Everything here is bound by reading the packed weights once. A workgroup owns one tile of 16 output
// channels (gated: the gate tile and the up tile of the same 16 activations); its waves split the K
// units between them and add their partial tiles through LDS in a fixed order.
#include <hip/hip_runtime.h>

#include "decode_ops.h"
#include "elementwise_ops.h"
#include "internal.h"

namespace hq {

namespace {

constexpr int kDecWaves = 8;

struct DecW {
  const uint8_t* w;
  size_t scales_off, zeros_off, expert_stride;
  int units;   // 128-k units per channel tile
  int asym;
};

template <int F>
__device__ __forceinline__ DecMeta<F> load_meta(const DecW& W, const uint8_t* w, int64_t nt, int u, int lane) {
  using T = DecTraits<F>;
  DecMeta<F> m;
  const size_t at = size_t(nt) * W.units + u;
  const int n = lane & 15;
  if constexpr (F == DF_G128) {
    m.s[0] = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(w + W.scales_off + at * 32 + 2 * n));
    uint32_t z = 8;
    if (W.asym) z = (w[W.zeros_off + at * 8 + (n >> 1)] >> (4 * (n & 1))) & 0xF;
    m.zo[0] = dec_zero_offset(z);
  } else if constexpr (T::kFine) {
    const uint8_t* b = w + W.scales_off + at * fine_meta_bytes(T::kG, W.asym);
#pragma unroll
    for (int g = 0; g < T::kGroups; ++g) {
      m.s[g] = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(b + (n * T::kGroups + g) * 2));
      uint32_t z = 8;
      if (W.asym) z = (b[fine_scale_bytes(T::kG) + n * (T::kGroups / 2) + (g >> 1)] >> (4 * (g & 1))) & 0xF;
      m.zo[g] = dec_zero_offset(z);
    }
  } else if constexpr (F == DF_MXFP4) {
    m.s[0] = e8m0_to_f32(w[W.scales_off + at * 64 + lane]);
    m.zo[0] = 0.f;
  } else {
    m.s[0] = m.zo[0] = 0.f;
  }
  return m;
}

// The channel's scale of 8-bit weights, 1 elsewhere.
template <int F>
__device__ __forceinline__ float channel_scale(const DecW& W, const uint8_t* w, int64_t n) {
  if constexpr (DecTraits<F>::kW8) return reinterpret_cast<const float*>(w + W.scales_off)[n];
  return 1.0f;
}

// This wave's share (units wave, wave + kDecWaves, ...) of row block x . tile nt of the expert at w.
// row: the lane's activation row (the MFMA's row lane & 15).
template <int F>
__device__ __forceinline__ void tile_product(float (&acc)[4], const DecW& W, const uint8_t* w, int64_t nt,
                                             const uint16_t* row, int wave, int lane) {
  using T = DecTraits<F>;
  for (int u = wave; u < W.units; u += kDecWaves) {
    const uint8_t* unit = w + (size_t(nt) * W.units + u) * T::kUnit;
    const u32x4 q0 = ldg16_stream(unit + 16 * lane);
    u32x4 q1 = {0u, 0u, 0u, 0u};
    if constexpr (T::kW8) q1 = ldg16_stream(unit + kUnitBytes + 16 * lane);
    u32x4 af[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) af[d] = ldg16(row + size_t(u) * 128 + 8 * dec_a_chunk<F>(lane >> 4, d));
    f32x4 rs[T::kGroups];
    dec_row_sums<F>(af, rs);
    dec_unit<F, 4>(acc, af, rs, q0, q1, load_meta<F>(W, w, nt, u, lane));
  }
}

// Sum of the waves' tiles: element i of a lane over the waves, in wave order. Returns thread
// (lane le, element i) pairs' sums for q = threadIdx.x < 256.
__device__ __forceinline__ float wave_tiles_sum(float (*red)[4][64], const float (&acc)[4], int wave, int lane, int q) {
  __syncthreads();   // the previous use has been read
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  float sum = 0.f;
  if (q < 256) {
    for (int v = 0; v < kDecWaves; ++v) sum += red[v][q >> 6][q & 63];
  }
  return sum;
}

struct GemvParams {
  DecW W;
  const uint16_t* x;
  uint16_t* y;
  int64_t M, N, K;   // N: weight rows (gated: 2 outputs' worth)
};

// Row block blockIdx.y, channel tile blockIdx.x.
template <int F, bool GATED>
__global__ __launch_bounds__(kDecWaves * 64) void gemv_kernel(GemvParams p) {
  __shared__ float red[kDecWaves][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = int64_t(blockIdx.y) * 16, nt = blockIdx.x;
  const int64_t outs = GATED ? p.N / 2 : p.N;
  const uint16_t* row = p.x + min(row0 + (lane & 15), p.M - 1) * p.K;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  tile_product<F>(acc, p.W, p.W.w, nt, row, wave, lane);
  float y = wave_tiles_sum(red, acc, wave, lane, threadIdx.x);
  const int le = threadIdx.x & 63;
  const int64_t n = nt * 16 + (le & 15), m = row0 + 4 * (le >> 4) + (threadIdx.x >> 6);
  const bool live = threadIdx.x < 256 && m < p.M;
  if (live) y *= channel_scale<F>(p.W, p.W.w, n);
  if constexpr (GATED) {
    float up[4] = {0.f, 0.f, 0.f, 0.f};
    tile_product<F>(up, p.W, p.W.w, nt + outs / 16, row, wave, lane);
    const float u = wave_tiles_sum(red, up, wave, lane, threadIdx.x);
    if (live) y = silu(y) * (u * channel_scale<F>(p.W, p.W.w, n + outs));
  }
  if (live) p.y[m * outs + n] = f32_to_bf16_rne(y);
}

struct MoeParams {
  DecW W;
  const uint16_t* x;      // gate_up: [T, K] tokens; down: [T * topk, K] activations
  const int32_t* ids;
  const float* weights;   // down
  uint16_t* y;            // gate_up: [T * topk, I]; down: [T, H]
  int topk, E;
  int64_t N, K;
};

// act[p] = silu(Wg x) * (Wu x) for routed entry p = blockIdx.y, 16 activations per workgroup.
template <int F>
__global__ __launch_bounds__(kDecWaves * 64) void moe_gate_up_kernel(MoeParams p) {
  __shared__ float red[kDecWaves][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int f = blockIdx.y;
  const int e = p.ids[f];
  if (e < 0 || e >= p.E) return;
  const uint8_t* w = p.W.w + size_t(e) * p.W.expert_stride;
  const uint16_t* row = p.x + int64_t(f / p.topk) * p.K;
  const int64_t nt = blockIdx.x, I = p.N / 2;
  float g[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
  tile_product<F>(g, p.W, w, nt, row, wave, lane);
  tile_product<F>(u, p.W, w, nt + I / 16, row, wave, lane);
  const float gs = wave_tiles_sum(red, g, wave, lane, threadIdx.x);
  const float us = wave_tiles_sum(red, u, wave, lane, threadIdx.x);
  if (threadIdx.x < 16) {
    const int64_t n = nt * 16 + threadIdx.x;
    const float a = silu(gs * channel_scale<F>(p.W, w, n)) * (us * channel_scale<F>(p.W, w, n + I));
    p.y[f * I + n] = f32_to_bf16_rne(a);
  }
}

// out[t] = sum over the token's routed entries of weight * Wd act, 16 outputs per workgroup.
template <int F>
__global__ __launch_bounds__(kDecWaves * 64) void moe_down_kernel(MoeParams p) {
  __shared__ float red[kDecWaves][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.y;
  const int64_t nt = blockIdx.x;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < p.topk; ++j) {
    const int f = t * p.topk + j;
    const int e = p.ids[f];
    if (e < 0 || e >= p.E) continue;
    const uint8_t* w = p.W.w + size_t(e) * p.W.expert_stride;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    tile_product<F>(a, p.W, w, nt, p.x + int64_t(f) * p.K, wave, lane);
    const float wt = (p.weights ? p.weights[f] : 1.0f) * channel_scale<F>(p.W, w, nt * 16 + (lane & 15));
    acc[0] = fmaf(wt, a[0], acc[0]);
  }
  const float y = wave_tiles_sum(red, acc, wave, lane, threadIdx.x);
  if (threadIdx.x < 16) p.y[t * p.N + nt * 16 + threadIdx.x] = f32_to_bf16_rne(y);
}

DecW dec_weights(const Combo& c, const uint8_t* w, int64_t N, int64_t K) {
  const PackedLayout L = c.fine_group ? make_fine_layout(c.fine_group, c.asym, N, K) : make_layout(c.fam, c.asym, N, K);
  return DecW{w, L.scales_off, L.zeros_off, L.expert_stride, int(K / 128), int(c.asym)};
}

int dec_format(const Combo& c) {
  if (c.fine_group) return c.fine_group == 32 ? DF_G32 : DF_G64;
  return c.fam == FAM_WNA16 ? DF_G128 : c.fam == FAM_MXW4A16 ? DF_MXFP4 : c.fam == FAM_W8A16 ? DF_INT8 : DF_FP8;
}

template <int F>
void gemv_fmt(const GemvCall& g, hipStream_t s) {
  GemvParams p{dec_weights(g.c, g.w, g.N, g.K), static_cast<const uint16_t*>(g.x), static_cast<uint16_t*>(g.y), g.M, g.N, g.K};
  const dim3 grid(unsigned(g.N / 16 / (g.gated ? 2 : 1)), unsigned((g.M + 15) / 16));
  if (g.gated)
    hipLaunchKernelGGL((gemv_kernel<F, true>), grid, dim3(kDecWaves * 64), 0, s, p);
  else
    hipLaunchKernelGGL((gemv_kernel<F, false>), grid, dim3(kDecWaves * 64), 0, s, p);
}

template <int F>
hipError_t moe_fmt(const MoeDecodeCall& m, hipStream_t s) {
  uint16_t* act = static_cast<uint16_t*>(m.ws);
  MoeParams up{dec_weights(m.c, m.w_gate_up, 2 * m.I, m.H), static_cast<const uint16_t*>(m.x), m.topk_ids, nullptr, act,
               m.topk, m.E, 2 * m.I, m.H};
  hipLaunchKernelGGL((moe_gate_up_kernel<F>), dim3(unsigned(m.I / 16), unsigned(m.T * m.topk)), dim3(kDecWaves * 64), 0, s, up);
  if (hipError_t e = hipGetLastError()) return e;
  MoeParams down{dec_weights(m.c, m.w_down, m.H, m.I), act, m.topk_ids, m.topk_weights, static_cast<uint16_t*>(m.out),
                 m.topk, m.E, m.H, m.I};
  hipLaunchKernelGGL((moe_down_kernel<F>), dim3(unsigned(m.H / 16), unsigned(m.T)), dim3(kDecWaves * 64), 0, s, down);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemv(const GemvCall& g, hipStream_t s) {
  switch (dec_format(g.c)) {
    case DF_G128: gemv_fmt<DF_G128>(g, s); break;
    case DF_G64: gemv_fmt<DF_G64>(g, s); break;
    case DF_G32: gemv_fmt<DF_G32>(g, s); break;
    case DF_MXFP4: gemv_fmt<DF_MXFP4>(g, s); break;
    case DF_INT8: gemv_fmt<DF_INT8>(g, s); break;
    default: gemv_fmt<DF_FP8>(g, s); break;
  }
  return hipGetLastError();
}

// The activations between the two launches, one bf16 row per routed entry.
size_t moe_decode_ws_bytes(const Combo&, int64_t T, int32_t topk, int32_t, int64_t, int64_t I) {
  return align256(size_t(T) * topk * I * 2);
}

hipError_t launch_moe_decode(const MoeDecodeCall& m, hipStream_t s) {
  switch (dec_format(m.c)) {
    case DF_G128: return moe_fmt<DF_G128>(m, s);
    case DF_G64: return moe_fmt<DF_G64>(m, s);
    case DF_G32: return moe_fmt<DF_G32>(m, s);
    case DF_MXFP4: return moe_fmt<DF_MXFP4>(m, s);
    case DF_INT8: return moe_fmt<DF_INT8>(m, s);
    default: return moe_fmt<DF_FP8>(m, s);
  }
}

}  // namespace hq
