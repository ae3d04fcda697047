// decode_ops.h -- one weight unit (16 channels x 128 k) of the decode calls: its operands, its
// dequantization and its MFMAs, for every weight format with bf16 activations that hq_gemv and
// hq_moe_decode take.
//
// A wave multiplies a row block (the MFMA's A operand: 1, up to 4, or up to 16 rows) by a unit.
// The result tile D leaves row 4 g + i, channel n in element i of lane 16 g + n, so with up to four
// rows the rows are placed at MFMA rows 0, 4, 8 and 12: row g is then element 0 of lane group g,
// and the per-group scaling (which the vector ALU does, next to the dequantization the largest
// share of its work) touches one element instead of four. The other MFMA rows repeat live ones and
// are dropped: rows do not mix in a matrix product.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_ops.h"
#include "layout.h"

namespace hq {

enum DecFmt { DF_G128 = 0, DF_G64 = 1, DF_G32 = 2, DF_MXFP4 = 3, DF_INT8 = 4, DF_FP8 = 5 };

template <int F>
struct DecTraits {
  static constexpr bool kInt4 = F == DF_G128 || F == DF_G64 || F == DF_G32;
  static constexpr bool kW8 = F == DF_INT8 || F == DF_FP8;
  static constexpr bool kFine = F == DF_G64 || F == DF_G32;
  static constexpr int kGroups = F == DF_G32 ? 4 : F == DF_G64 ? 2 : 1;   // scale groups per unit (INT4)
  static constexpr int kG = 128 / kGroups;
  static constexpr int kWLoads = kW8 ? 2 : 1;        // 1 KiB of codes each
  static constexpr int kUnit = kUnitBytes * kWLoads; // code bytes of 16 channels x 128 k
};

// Which 16-byte chunk (8 k) of a unit's 128 k lane group g feeds to MFMA d: the k order of the
// format's prepacked codes (layout.h).
template <int F>
__device__ __forceinline__ constexpr int dec_a_chunk(int g, int d) {
  return DecTraits<F>::kFine ? 4 * d + g : 4 * g + d;
}

// A unit's scales (and zeros) as lane l needs them, for channel l & 15.
template <int F>
struct DecMeta {
  float s[DecTraits<F>::kGroups];
  float zo[DecTraits<F>::kGroups];   // 128 + z
};

// 128 + z for a 4-bit z: 128.0's mantissa step at bit 16 is 1.
__device__ __forceinline__ float dec_zero_offset(uint32_t z) { return __uint_as_float(0x43000000u | (z << 16)); }

// acc += the unit's product. af: the A operand of MFMAs 0..3; q0 / q1: the lane's codes (q1: the
// second KiB of 8-bit weights). NE = 1: the rows stand at element 0 (see above); 4: all 16 rows.
//
// INT4: sum_k x (q - z) of a group is formed as sum_k x (128 + q) -- 128 + q is one bit-select per
// pair of codes, exact in bf16 -- less (128 + z) sum_k x, the row sums rs coming from the MFMA
// against ones (shared by a wave's tiles). Scales multiply the fp32 partial sum of each group:
// folded into the bf16 operand they would be rounded once per weight (2^-9 each).
template <int F, int NE>
__device__ __forceinline__ void dec_unit(float (&acc)[NE], const u32x4 (&af)[4], const f32x4 (&rs)[DecTraits<F>::kGroups],
                                         const u32x4& q0, const u32x4& q1, const DecMeta<F>& m) {
  using T = DecTraits<F>;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  if constexpr (T::kInt4) {
    constexpr int per = 4 / T::kGroups;   // MFMAs per group
#pragma unroll
    for (int g = 0; g < T::kGroups; ++g) {
      f32x4 part = zero;
#pragma unroll
      for (int d = g * per; d < (g + 1) * per; ++d)
        part = mfma_bf16(__builtin_bit_cast(bf16x8, af[d]), dequant_int4x8_offset128(q0[d]), part);
#pragma unroll
      for (int i = 0; i < NE; ++i) acc[i] = fmaf(m.s[g], fmaf(-m.zo[g], rs[g][i], part[i]), acc[i]);
    }
  } else {
    f32x4 part = zero;
#pragma unroll
    for (int i = 0; i < NE; ++i) part[i] = acc[i];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      bf16x8 b;
      if constexpr (F == DF_MXFP4) b = dequant_fp4x8_scaled(q0[d], m.s[0]);
      else b = dequant_w8_step<F == DF_FP8>(q0, q1, d);
      part = mfma_bf16(__builtin_bit_cast(bf16x8, af[d]), b, part);
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) acc[i] = part[i];
  }
}

// Row sums of the unit's groups (INT4 only): the A operand against ones.
template <int F>
__device__ __forceinline__ void dec_row_sums(const u32x4 (&af)[4], f32x4 (&rs)[DecTraits<F>::kGroups]) {
  using T = DecTraits<F>;
  if constexpr (T::kInt4) {
    const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
    constexpr int per = 4 / T::kGroups;
#pragma unroll
    for (int g = 0; g < T::kGroups; ++g) {
      rs[g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = g * per; d < (g + 1) * per; ++d) rs[g] = mfma_bf16(__builtin_bit_cast(bf16x8, af[d]), ones, rs[g]);
    }
  }
}

}  // namespace hq
