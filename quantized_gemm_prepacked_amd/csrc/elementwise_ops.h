// elementwise_ops.h -- device helpers shared by the MoE layer's elementwise kernels and the
// quantizers of activations, norms and caches (the gated activation feeds a quantizer when the Down GEMM takes
// 8-bit activations, and both paths must produce the same bits).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hq {

// silu(g) = g * sigmoid(g), with sigmoid(g) = 1 / (1 + e) for g >= 0 and e / (1 + e) for g < 0,
// e = exp(-|g|): e never overflows, so a very negative gate keeps its tiny product instead of
// dividing by an infinite exp(-g).
__device__ __forceinline__ float silu(float g) {
  const float e = expf(-fabsf(g));
  return g * ((g >= 0.0f ? 1.0f : e) / (1.0f + e));
}

// fp32(v / s), the IEEE quotient, from rs = fp32(1 / s): a product and two corrections by the exact
// remainder, six operations where the compiler's division takes about twelve. After the first correction
// the quotient is within one unit in its last place, after the second it is rounded correctly (Markstein's
// theorem: a correctly rounded reciprocal, an exact remainder). That holds while neither reciprocal nor
// remainder leaves the normal range; scales outside 2^-80 .. 2^80 take the division. Remainders of quotients
// below 2^-20 or so may be inexact: those codes are 0 either way. The corrections turn -0 into 0: the sign is put back.
__device__ __forceinline__ float quotient(float v, float s, float rs) {
  if (!(s > 0x1p-80f && s < 0x1p80f)) return v / s;
  float q = v * rs;
  q = fmaf(fmaf(-q, s, v), rs, q);
  return copysignf(fmaf(fmaf(-q, s, v), rs, q), v);
}

// Four codes of values in units of their scale, one a byte. e4m3: nearest code, ties to even, saturating
// at 448 (gfx950's conversion of a clamped value); the sign stays on a zero. INT8: rounded half to even,
// then clamped to +-127.
__device__ __forceinline__ uint32_t e4m3x4_rne(float a, float b, float c, float d) {
  const auto m = [](float v) { return __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f); };
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(m(a), m(b), 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(m(c), m(d), lo, true));
}
__device__ __forceinline__ uint32_t int8_rne(float v) {
  return uint32_t(int(__builtin_amdgcn_fmed3f(__builtin_rintf(v), -127.0f, 127.0f))) & 0xFFu;
}
__device__ __forceinline__ uint32_t int8x4_rne(float a, float b, float c, float d) {
  return int8_rne(a) | (int8_rne(b) << 8) | (int8_rne(c) << 16) | (int8_rne(d) << 24);
}

// e2m1 magnitude code of a >= 0 (exact binary32), ties to the even code, saturating at 6.
__device__ __forceinline__ uint32_t e2m1_code(float a) {
  return uint32_t(a > 0.25f) + uint32_t(a >= 0.75f) + uint32_t(a > 1.25f) + uint32_t(a >= 1.75f) +
         uint32_t(a > 2.5f) + uint32_t(a >= 3.5f) + uint32_t(a > 5.0f);
}

}  // namespace hq
