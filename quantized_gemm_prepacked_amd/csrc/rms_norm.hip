// rms_norm.hip -- RMS norm with the residual's addition in front and the activation quantization of
// the following GEMM behind: h = bf16(x + residual), v = (h * r) * weight with r = 1 / sqrt(mean h^2 +
// eps), written as bf16 or as codes and scales by the rules of act_quant.hip, applied to the unrounded v.
//
// The sum of squares is in binary64. Squares of bf16 values are exact there, and a sum has 86 roundings at most (64 terms a thread, 6 and 16
// joins): two orders of it, for another number of threads, differ by less than 2 * 86 * 2^-53 of it, and r, rounded to 2^-24, differs in
// fewer than one row of a million. The conversion and the add run at the vector units' ordinary rate, far below what the loads take.
//
// A row is held in registers between its passes (sum, maximum, codes): each thread keeps C chunks of
// eight bf16 sums h, so memory is read and written once. What bounds it is that traffic: 8192 rows of
// 8192 to INT8 with a residual move 470 MB in 86 us, 5.5 TB/s, where a copy reaches 5.0. One row of
// 4096 takes 3.6 us to e4m3, a launch, two dependent trips to memory and two reductions. Rows past 32768 columns are 8 chunks a thread, which spill
// 15 to 28 registers: 512 of 40960 to INT8 61 us, 2.4 TB/s (of 32768, 4 chunks: 34 us, 3.4 TB/s).
#include <hip/hip_runtime.h>

#include "device_ops.h"
#include "elementwise_ops.h"
#include "internal.h"

namespace hq {

namespace {

__device__ __forceinline__ float bf16_at(const u32x4& v, int j) {
  return __uint_as_float((j & 1) ? (v[j >> 1] & 0xFFFF0000u) : (v[j >> 1] << 16));
}

// Sum (binary64) or maximum over the TPR threads of a row: within the wave by shuffles, over the
// workgroup's waves through LDS. `slot` is scratch that this reduction alone uses between two barriers.
template <int TPR, class T, class F>
__device__ __forceinline__ T row_reduce(T v, T* slot, F join) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = join(v, __shfl_xor(v, off, 64));
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v = join(v, slot[w]);
  }
  return v;
}

// The scale of a row or block whose largest |v| is amax.
template <int ACT>
__device__ __forceinline__ float scale_of(float amax) {
  const float s = amax * (ACT == HQ_ACT_INT8_PER_TOKEN ? 1.0f / 127.0f : 1.0f / 448.0f);
  return s == 0.0f ? 1.0f : s;
}

// Eight codes of v[0..7] at scale s (rs = 1 / s), as two dwords.
template <int ACT>
__device__ __forceinline__ uint2 codes8(const float* v, float s, float rs) {
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = quotient(v[j], s, rs);
  uint2 out;
  if constexpr (ACT == HQ_ACT_INT8_PER_TOKEN) {
    out.x = int8x4_rne(q[0], q[1], q[2], q[3]);
    out.y = int8x4_rne(q[4], q[5], q[6], q[7]);
  } else {
    out.x = e4m3x4_rne(q[0], q[1], q[2], q[3]);
    out.y = e4m3x4_rne(q[4], q[5], q[6], q[7]);
  }
  return out;
}

// TPR threads a row, C chunks of TPR * 8 columns.
template <int ACT, int TPR, int C>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rms_norm_kernel(RmsNormCall a) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;   // rows a workgroup
  constexpr bool kRowScale = ACT == HQ_ACT_INT8_PER_TOKEN || ACT == HQ_ACT_FP8E4M3_PER_TOKEN;
  __shared__ double sums[TPR / 64];
  __shared__ float tops[TPR / 64];
  const int tid = threadIdx.x % TPR;
  const int K = int(a.K);
  const auto* weight = static_cast<const uint16_t*>(a.weight);
  for (int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / TPR; row < a.M; row += int64_t(gridDim.x) * kRows) {
    const size_t at = size_t(row) * K;
    const auto* x = static_cast<const uint16_t*>(a.x) + at;
    u32x4 h[C], w[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * TPR + tid) * 8;
      h[c] = i < K ? ldg16(x + i) : u32x4{0, 0, 0, 0};
    }
    if (a.residual) {
      const auto* r = static_cast<const uint16_t*>(a.residual) + at;
      auto* ro = static_cast<uint16_t*>(a.residual_out) + at;
      u32x4 add[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = (c * TPR + tid) * 8;
        add[c] = i < K ? ldg16(r + i) : u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = (c * TPR + tid) * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[c][j] = f32x2_to_bf16x2_rne(bf16_at(h[c], 2 * j) + bf16_at(add[c], 2 * j), bf16_at(h[c], 2 * j + 1) + bf16_at(add[c], 2 * j + 1));
        if (i < K) *reinterpret_cast<u32x4*>(ro + i) = h[c];
      }
    }
    // asked for before the sum is needed
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * TPR + tid) * 8;
      w[c] = weight && i < K ? ldg16(weight + i) : u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    }
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double d = double(bf16_at(h[c], j));
        sum = fma(d, d, sum);
      }
    sum = row_reduce<TPR>(sum, sums, [](double p, double q) { return p + q; });
    const float r = float(1.0 / sqrt(sum / double(K) + double(a.eps)));
    const auto v8 = [&](int c, float* v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (bf16_at(h[c], j) * r) * bf16_at(w[c], j);
    };
    float s = 1.0f;
    if constexpr (kRowScale) {
      float amax = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float v[8];
        v8(c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
      }
      s = scale_of<ACT>(row_reduce<TPR>(amax, tops, [](float p, float q) { return fmaxf(p, q); }));
      if (tid == 0) static_cast<float*>(a.y_scale)[row] = s;
    }
    const float rs = 1.0f / s;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * TPR + tid) * 8;
      float v[8];
      v8(c, v);
      float amax = 0.0f;
      if constexpr (!kRowScale && ACT != HQ_ACT_BF16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
        // the 16 (block of 128) or 4 (MX block) lanes that share a scale: all of them are within K, or none
#pragma unroll
        for (int off = ACT == HQ_ACT_FP8E4M3_BLOCK128 ? 8 : 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
      }
      if (i >= K) continue;
      if (ACT == HQ_ACT_BF16 || a.y_bf16) {
        const u32x4 b = {f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3]), f32x2_to_bf16x2_rne(v[4], v[5]),
                         f32x2_to_bf16x2_rne(v[6], v[7])};
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(ACT == HQ_ACT_BF16 ? a.y : a.y_bf16) + at + i) = b;
      }
      auto* y = static_cast<uint8_t*>(a.y) + (ACT == HQ_ACT_MXFP4 ? (at + i) / 2 : at + i);
      if constexpr (kRowScale) {
        *reinterpret_cast<uint2*>(y) = codes8<ACT>(v, s, rs);
      } else if constexpr (ACT == HQ_ACT_FP8E4M3_BLOCK128) {
        const float sb = scale_of<ACT>(amax);
        if ((tid & 15) == 0) static_cast<float*>(a.y_scale)[(at + i) >> 7] = sb;
        *reinterpret_cast<uint2*>(y) = codes8<ACT>(v, sb, 1.0f / sb);
      } else if constexpr (ACT == HQ_ACT_MXFP8 || ACT == HQ_ACT_MXFP4) {
        // e = floor(log2 amax) - the elements' largest exponent, from the bits; a subnormal amax counts as 0
        const int ef = int(__float_as_uint(amax) >> 23);
        const int e = ef == 0 ? -127 : max(ef - 127 - (ACT == HQ_ACT_MXFP8 ? 8 : 2), -127);
        if ((tid & 3) == 0) static_cast<uint8_t*>(a.y_scale)[(at + i) >> 5] = uint8_t(e + 127);
        const float up = __uint_as_float(uint32_t(127 - e) << 23);   // 2^-e: e is -127 .. 125
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= up;
        if constexpr (ACT == HQ_ACT_MXFP8) {
          *reinterpret_cast<uint2*>(y) = make_uint2(e4m3x4_rne(v[0], v[1], v[2], v[3]), e4m3x4_rne(v[4], v[5], v[6], v[7]));
        } else {
          uint32_t word = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t code = e2m1_code(fabsf(v[j]));
            word |= (code | uint32_t(v[j] < 0.0f && code != 0u) << 3) << (4 * j);
          }
          *reinterpret_cast<uint32_t*>(y) = word;
        }
      }
    }
    // the next row's reductions write the scratch that this row's threads may still read
    if constexpr (TPR > 64) __syncthreads();
  }
}

template <int ACT, int TPR, int C>
hipError_t go(const RmsNormCall& a, hipStream_t s) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  const int64_t groups = (a.M + kRows - 1) / kRows;
  const dim3 grid(unsigned(groups < (1 << 20) ? groups : 1 << 20));
  hipLaunchKernelGGL((rms_norm_kernel<ACT, TPR, C>), grid, dim3(TPR < 256 ? 256 : TPR), 0, s, a);
  return hipGetLastError();
}

// Threads a row. Few rows leave most of the chip idle, so a row's latency counts and more threads with less each are better;
// with many rows the loads in flight count, and the idle threads behind the row's end. Measured with a residual, in us:
//   K 2048, INT8:    64 threads 5.4 at 67 rows, 6.6 at 1024, 14.6 at 4099; 256 threads 4.1, 6.9, 17.0
//   K 4096, INT8:    256 threads 4.4 at 1 row, 5.1 at 256, 6.5 at 512, 26.6 at 4099; 512 threads 4.3, 5.1, 7.1, 31.6; 64 threads 6.9, 8.0, 8.8, 30.7
//   K 8192, MXFP8:   256 threads 4.8 at 67 rows, 9.2 at 512, 26.6 at 2048, 46.5 at 4099; 512 threads 4.4, 9.0, 29.8, 52.1
//   K 8192, INT8:    256 threads 6.1 at 67 rows, 10.4 at 512, 14.8 at 1024; 512 threads 5.3, 10.0, 14.5
//   K 14336, INT8:   512 threads 6.7 at 67 rows, 79.4 at 4099; 1024 threads 6.5, 79.9; 256 threads 8.0, 81.2
template <int ACT>
hipError_t pick(const RmsNormCall& a, hipStream_t s) {
  const bool many = a.M >= 1024;
  if (a.K <= 512) return go<ACT, 64, 1>(a, s);
  if (a.K <= 1024) return go<ACT, 64, 2>(a, s);
  if (a.K <= 2048) return many ? go<ACT, 64, 4>(a, s) : go<ACT, 256, 1>(a, s);
  if (a.K <= 4096) return a.M <= 256 ? go<ACT, 512, 1>(a, s) : go<ACT, 256, 2>(a, s);
  if (a.K <= 8192) {
    if (!many) return go<ACT, 512, 2>(a, s);
    return a.K <= 6144 ? go<ACT, 256, 3>(a, s) : go<ACT, 256, 4>(a, s);
  }
  if (a.K <= 16384) return go<ACT, 1024, 2>(a, s);
  if (a.K <= 32768) return go<ACT, 1024, 4>(a, s);
  return go<ACT, 1024, 8>(a, s);
}

}  // namespace

hipError_t launch_rms_norm(const RmsNormCall& a, hipStream_t s) {
  switch (a.act_fmt) {
    case HQ_ACT_BF16: return pick<HQ_ACT_BF16>(a, s);
    case HQ_ACT_INT8_PER_TOKEN: return pick<HQ_ACT_INT8_PER_TOKEN>(a, s);
    case HQ_ACT_FP8E4M3_PER_TOKEN: return pick<HQ_ACT_FP8E4M3_PER_TOKEN>(a, s);
    case HQ_ACT_FP8E4M3_BLOCK128: return pick<HQ_ACT_FP8E4M3_BLOCK128>(a, s);
    case HQ_ACT_MXFP8: return pick<HQ_ACT_MXFP8>(a, s);
    default: return pick<HQ_ACT_MXFP4>(a, s);
  }
}

}  // namespace hq
