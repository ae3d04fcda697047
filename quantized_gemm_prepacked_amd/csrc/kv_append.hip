// kv_append.hip -- new keys and values quantized into the paged cache: one scale a page and head.
//
// One workgroup takes one touched page of one sequence, one head, K or V: the largest magnitude of the
// page's new tokens, the page's scale (a new one, or the held one times a power of two), the codes of the
// new tokens, and where the scale grew the codes that were there. Nothing is shared between workgroups.
#include <hip/hip_runtime.h>

#include "device_ops.h"
#include "elementwise_ops.h"
#include "internal.h"
#include "kv_cache.h"

namespace hq {

namespace {

// Magnitude bits of a bf16 as the scale counts it: infinity as the largest finite value, NaN as nothing.
__device__ __forceinline__ uint32_t counted(uint32_t h) {
  const uint32_t m = h & 0x7FFFu;
  return m > 0x7F80u ? 0u : min(m, 0x7F7Fu);
}

// The code of a bf16 value at scale s (rs = 1 / s; s = 0: code 0); NaN gives `nan`.
template <int FMT>
__device__ __forceinline__ uint32_t code_of(uint32_t h, float s, float rs, uint32_t nan) {
  if ((h & 0x7FFFu) > 0x7F80u) return nan;
  const float v = __uint_as_float(((h & 0x8000u) | counted(h)) << 16);
  const float q = s == 0.0f ? 0.0f : quotient(v, s, rs);
  if constexpr (FMT == HQ_KV_INT8) return int8_rne(q);
  else return e4m3x4_rne(q, 0.0f, 0.0f, 0.0f) & 0xFFu;
}

// A code at 2^e times its scale; an e4m3 NaN stays one.
template <int FMT>
__device__ __forceinline__ uint32_t regrown(uint32_t code, float down) {
  if constexpr (FMT == HQ_KV_INT8) {
    return int8_rne(float(int8_t(code)) * down);
  } else {
    if ((code & 0x7Fu) == 0x7Fu) return code;
    return e4m3x4_rne(__builtin_amdgcn_cvt_f32_fp8(int(code), 0) * down, 0.0f, 0.0f, 0.0f) & 0xFFu;
  }
}

template <int FMT, int THREADS>
__global__ __launch_bounds__(THREADS) void kv_append_kernel(KvCall c) {
  constexpr float kUnit = FMT == HQ_KV_INT8 ? 1.0f / 127.0f : 1.0f / 448.0f;
  const int b = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int head = int(blockIdx.x % unsigned(c.H));
  const KvSeq q = kv_sequence(c, b);
  const int P = 1 << c.page_shift, D = c.D;
  const int begin = max(q.len - q.n, 0);                 // first position stored
  const int page_at = (begin >> c.page_shift) + int(blockIdx.x / unsigned(c.H));
  const int lo = max(begin, page_at << c.page_shift), hi = min(q.len, (page_at + 1) << c.page_shift);
  if (q.n == 0 || lo >= hi) return;
  const int page = c.table[int64_t(b) * c.width + page_at];
  if (page < 0 || page >= c.num_pages) return;
  const int slot0 = lo & (P - 1), count = hi - lo;
  // row of position p: first + p - (len - n)
  const auto* src = static_cast<const uint16_t*>(is_v ? c.v : c.k) + (int64_t(q.first) + lo - (q.len - q.n)) * c.kv_stride + int64_t(head) * D;
  uint8_t* dst = static_cast<uint8_t*>(is_v ? c.v_pages : c.k_pages) + (int64_t(page) * c.H + head) * (int64_t(P) * D);
  float* scale = (is_v ? c.v_scales : c.k_scales) + int64_t(page) * c.H + head;
  const int chunks = D / 8;

  uint32_t top = 0;
  for (int i = threadIdx.x; i < count * chunks; i += THREADS) {
    const u32x4 x = ldg16(src + (i / chunks) * c.kv_stride + (i % chunks) * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, max(counted(x[j] & 0xFFFFu), counted(x[j] >> 16)));
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = max(top, uint32_t(__shfl_xor(int(top), off, 64)));
  if constexpr (THREADS > 64) {
    __shared__ uint32_t tops[THREADS / 64];
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) top = max(top, tops[w]);
  }
  const float need = __uint_as_float(top << 16) * kUnit;
  float s = need, down = 1.0f;
  if (slot0 != 0) {
    const float held = *scale;
    if (held != 0.0f) {
      s = held;
      if (need > held) {
        int en, eh;
        const float mn = frexpf(need, &en), mh = frexpf(held, &eh);
        const int e = en - eh + (mn > mh ? 1 : 0);
        s = ldexpf(held, e);
        down = ldexpf(1.0f, -e);
      }
    }
  }
  // every thread has read the held scale before one writes it
  if constexpr (THREADS > 64) __syncthreads();
  if (threadIdx.x == 0) *scale = s;
  const float rs = 1.0f / s;

  if (!is_v) {
    const uint32_t nan = FMT == HQ_KV_INT8 ? 0u : 0x7Fu;
    if (down != 1.0f)
      for (int i = threadIdx.x; i < slot0 * D / 4; i += THREADS) {
        uint32_t* at = reinterpret_cast<uint32_t*>(dst) + i;
        uint32_t w = *at, out = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) out |= regrown<FMT>((w >> (8 * j)) & 0xFFu, down) << (8 * j);
        *at = out;
      }
    for (int i = threadIdx.x; i < count * chunks; i += THREADS) {
      const u32x4 x = ldg16(src + (i / chunks) * c.kv_stride + (i % chunks) * 8);
      uint2 out = {0u, 0u};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        out.x |= code_of<FMT>((x[j >> 1] >> (16 * (j & 1))) & 0xFFFFu, s, rs, nan) << (8 * j);
        out.y |= code_of<FMT>((x[2 + (j >> 1)] >> (16 * (j & 1))) & 0xFFFFu, s, rs, nan) << (8 * j);
      }
      *reinterpret_cast<uint2*>(dst + (int64_t(slot0) * chunks + i) * 8) = out;
    }
  } else {
    if (down != 1.0f)
      for (int i = threadIdx.x; i < slot0 * D; i += THREADS) {
        uint8_t* at = dst + (i / slot0) * P + i % slot0;
        *at = uint8_t(regrown<FMT>(*at, down));
      }
    // four slots of eight channels a thread: whole dwords where all four slots are new, bytes at the ends
    const int quad0 = slot0 >> 2, quads = ((slot0 + count - 1) >> 2) - quad0 + 1;
    for (int i = threadIdx.x; i < quads * chunks; i += THREADS) {
      const int at = (quad0 + i / chunks) * 4, d0 = (i % chunks) * 8;
      uint32_t word[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int token = at + t - slot0;
        if (token < 0 || token >= count) continue;
        const u32x4 x = ldg16(src + token * c.kv_stride + d0);
#pragma unroll
        for (int j = 0; j < 8; ++j) word[j] |= code_of<FMT>((x[j >> 1] >> (16 * (j & 1))) & 0xFFFFu, s, rs, 0u) << (8 * t);
      }
      const bool whole = at >= slot0 && at + 4 <= slot0 + count;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint8_t* to = dst + int64_t(d0 + j) * P + at;
        if (whole) {
          *reinterpret_cast<uint32_t*>(to) = word[j];
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (at + t >= slot0 && at + t < slot0 + count) to[t] = uint8_t(word[j] >> (8 * t));
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const KvCall& c, hipStream_t s) {
  const int64_t pages = ((int64_t(c.max_new) + (1 << c.page_shift) - 2) >> c.page_shift) + 1;   // at most, of a sequence
  const dim3 grid(unsigned(pages * c.H), unsigned(c.B), 2u);
  if (c.fmt == HQ_KV_INT8) hipLaunchKernelGGL((kv_append_kernel<HQ_KV_INT8, 256>), grid, dim3(256), 0, s, c);
  else hipLaunchKernelGGL((kv_append_kernel<HQ_KV_FP8_E4M3, 256>), grid, dim3(256), 0, s, c);
  return hipGetLastError();
}

}  // namespace hq
