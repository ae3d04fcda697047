// kv_append.hip -- new keys and values quantized into the paged cache: one scale a page and head.
//
// One workgroup (one wave where there are only a few new tokens) takes one touched page of one sequence, one head, K or V: the largest
// magnitude of the page's new tokens, the page's scale (a new one, or the held one times a power of two), the codes of the
// new tokens, and where the scale grew the codes that were there. Nothing is shared between workgroups.
//
// What bounds it is the traffic, each new value read once and each code written once: 5 prompts of up to 4000 tokens (INT8, 8
// heads of 128, 108 MB) take 25 us, 4.3 TB/s; one token of each of 48 sequences 4.5 us, a launch and the dependent
// reads of lengths, page, scale and tokens. Where a page's scale grows, its codes go through one wave (a few new tokens) or workgroup
// one dword (keys) or byte (values) a thread after another: 48 e4m3 tokens into pages of 16 / 64 / 256 slots of 128 channels 9 / 29 / 138 us, where
// they fit 3.4 / 3.8 / 3.8.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_ops.h"
#include "elementwise_ops.h"
#include "internal.h"
#include "kv_cache.h"

namespace hq {

namespace {

constexpr int kFewTokens = 4;     // new tokens of a sequence that one wave takes

// Magnitude bits of a bf16 as the scale counts it: infinity as the largest finite value, NaN as nothing.
__device__ __forceinline__ uint32_t counted(uint32_t h) {
  const uint32_t m = h & 0x7FFFu;
  return m > 0x7F80u ? 0u : min(m, 0x7F7Fu);
}

// fp32(v / s) of a bf16 v, from rs = fp32(1 / s): a product and one correction by the remainder. A bf16 has 128 mantissas and
// a scale, which may come from a page that was filled elsewhere, 2^23: the result is the IEEE quotient for every pair (all 2^30 tried on
// a CPU).
__device__ __forceinline__ float page_quotient(float v, float s, float rs) {
  const float q = v * rs;
  return fmaf(fmaf(-q, s, v), rs, q);
}

// Codes of the two bf16 in w, as bytes of (lo, hi). PLAIN: finite values within the scale, of a normal size.
template <int FMT, bool PLAIN>
__device__ __forceinline__ uint2 codes_of(uint32_t w, float s, float rs, uint32_t nan) {
  if constexpr (PLAIN) {
    const float a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xFFFF0000u);
    const float x = page_quotient(a, s, rs), y = page_quotient(b, s, rs);
    if constexpr (FMT == HQ_KV_INT8)      // 1.5 * 2^23 + q: rounded half to even, the code in the low byte
      return make_uint2(__float_as_uint(x + 12582912.0f), __float_as_uint(y + 12582912.0f));
    else {      // (the correction turns -0 into 0)
      const uint32_t c = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(copysignf(x, a), copysignf(y, b), 0, false));
      return make_uint2(c, c >> 8);
    }
  } else {
    const auto one = [&](uint32_t h) {
      if ((h & 0x7FFFu) > 0x7F80u) return nan;
      const float v = __uint_as_float(((h & 0x8000u) | counted(h)) << 16);
      const float q = s == 0.0f ? 0.0f : v / s;
      if constexpr (FMT == HQ_KV_INT8) return int8_rne(q);
      else return e4m3x4_rne(q, 0.0f, 0.0f, 0.0f);
    };
    return make_uint2(one(w & 0xFFFFu), one(w >> 16));
  }
}

// The low bytes of four words, as one.
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
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

// Items of a page: a key's chunk of eight channels, or four slots of eight channels of values, which become whole dwords of the
// transposed page. A thread's first kKeep items stay in registers between the pass that finds the largest magnitude and
// the pass that writes the codes; further ones (long pages of wide heads) are read again, from the caches.
template <int FMT, int D, int THREADS, bool V>
__device__ __forceinline__ void append_page(const uint16_t* src, int64_t stride, uint8_t* dst, float* scale, int shift, int slot0, int count) {
  constexpr float kUnit = FMT == HQ_KV_INT8 ? 1.0f / 127.0f : 1.0f / 448.0f;
  constexpr int kChunks = D / 8, kLoads = V ? 4 : 1, kKeep = V ? 1 : 4;
  const int P = 1 << shift;
  // Values go by quads of slots. A few tokens: chunks next to each other. A page: lanes next to each other take quads next to each other,
  // whose codes are, and all of the page's, a power of two.
  const int quad0 = slot0 >> 2, quads = ((slot0 + count + 3) >> 2) - quad0;
  const int items = !V ? count * kChunks : THREADS == 64 ? quads * kChunks : (P >> 2) * kChunks;
  const auto chunk_of = [&](int item) { return V && THREADS > 64 ? item >> (shift - 2) : item % kChunks; };
  const auto token_of = [&](int item) {
    return !V ? item / kChunks : THREADS == 64 ? 4 * (item / kChunks + quad0) - slot0 : 4 * (item & ((P >> 2) - 1)) - slot0;
  };
  const auto load = [&](int item, u32x4 (&x)[kLoads]) {
    const int c = chunk_of(item), t = token_of(item);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) x[k] = t + k >= 0 && t + k < count ? ldg16(src + (t + k) * stride + 8 * c) : u32x4{0, 0, 0, 0};
  };
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const auto largest = [](u16x2 top, const u32x4 (&x)[kLoads]) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x[k][j] & 0x7FFF7FFFu));
    return top;
  };
  const float held = slot0 != 0 ? *scale : 0.0f;      // (asked for with the items)
  u32x4 kept[kKeep][kLoads];
  u16x2 both = {0, 0};
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int item = threadIdx.x + k * THREADS;
    if (item < items) load(item, kept[k]);
    else
#pragma unroll
      for (int l = 0; l < kLoads; ++l) kept[k][l] = u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int k = 0; k < kKeep; ++k) both = largest(both, kept[k]);
  for (int item = threadIdx.x + kKeep * THREADS; item < items; item += THREADS) {
    u32x4 x[kLoads];
    load(item, x);
    both = largest(both, x);
  }
  const auto over_threads = [](uint32_t v, uint32_t* slots) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = max(v, uint32_t(__shfl_xor(int(v), off, 64)));
    if constexpr (THREADS > 64) {
      if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
      __syncthreads();      // (every thread has read the held scale before one writes it, too)
#pragma unroll
      for (int w = 0; w < THREADS / 64; ++w) v = max(v, slots[w]);
    }
    return v;
  };
  __shared__ uint32_t slots[2][THREADS / 64];
  uint32_t top = over_threads(max(uint32_t(both[0]), uint32_t(both[1])), slots[0]);
  const bool finite = top <= 0x7F7Fu;
  if (!finite) {      // infinities or NaN among them: counted one by one
    top = 0;
    for (int item = threadIdx.x; item < items; item += THREADS) {
      u32x4 x[kLoads];
      load(item, x);
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(counted(x[k][j] & 0xFFFFu), counted(x[k][j] >> 16)));
    }
    top = over_threads(top, slots[1]);
  }
  const float need = __uint_as_float(top << 16) * kUnit;
  float s = need, down = 1.0f;
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
  if (threadIdx.x == 0) *scale = s;
  const float rs = 1.0f / s;
  if (down != 1.0f) {      // the codes that were there
    if constexpr (V) {
      for (int i = threadIdx.x; i < slot0 * D; i += THREADS) {
        uint8_t* at = dst + (i / slot0) * P + i % slot0;
        *at = uint8_t(regrown<FMT>(*at, down));
      }
    } else {
      for (int i = threadIdx.x; i < slot0 * D / 4; i += THREADS) {
        uint32_t* at = reinterpret_cast<uint32_t*>(dst) + i;
        const uint32_t w = *at;
        uint32_t out = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) out |= regrown<FMT>((w >> (8 * j)) & 0xFFu, down) << (8 * j);
        *at = out;
      }
    }
  }
  const auto write = [&](const u32x4 (&x)[kLoads], int item, auto plain) {
    constexpr bool kPlain = decltype(plain)::value;
    const int c = chunk_of(item), t = token_of(item);
    if constexpr (V) {
      uint32_t word[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint2 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = codes_of<FMT, kPlain>(x[k][j], s, rs, 0u);
        word[2 * j] = bytes4(v[0].x, v[1].x, v[2].x, v[3].x);
        word[2 * j + 1] = bytes4(v[0].y, v[1].y, v[2].y, v[3].y);
      }
      uint8_t* to = dst + int64_t(8 * c) * P + slot0 + t;
      if (t >= 0 && t + 4 <= count) {
#pragma unroll
        for (int j = 0; j < 8; ++j) *reinterpret_cast<uint32_t*>(to + j * P) = word[j];
      } else {      // the slots at the ends, a byte each
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (t + k >= 0 && t + k < count)
#pragma unroll
            for (int j = 0; j < 8; ++j) to[j * P + k] = uint8_t(word[j] >> (8 * k));
      }
    } else {
      uint2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = codes_of<FMT, kPlain>(x[0][j], s, rs, FMT == HQ_KV_INT8 ? 0u : 0x7Fu);
      *reinterpret_cast<uint2*>(dst + int64_t(slot0 + t) * D + 8 * c) =
          make_uint2(bytes4(v[0].x, v[0].y, v[1].x, v[1].y), bytes4(v[2].x, v[2].y, v[3].x, v[3].y));
    }
  };
  const auto write_all = [&](auto plain) {
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const int item = threadIdx.x + k * THREADS;
      if (item < items) write(kept[k], item, plain);
    }
    for (int item = threadIdx.x + kKeep * THREADS; item < items; item += THREADS) {
      u32x4 x[kLoads];
      load(item, x);
      write(x, item, plain);
    }
  };
  // (the same for all threads)
  if (finite && s > 0x1p-80f && s < 0x1p80f) write_all(std::true_type{});
  else write_all(std::false_type{});
}

template <int FMT, int D, int THREADS>
__global__ __launch_bounds__(THREADS) void kv_append_kernel(KvCall c) {
  const int b = blockIdx.y;
  const int head = int(blockIdx.x % unsigned(c.H));
  const KvSeq q = kv_sequence(c, b);
  const int P = 1 << c.page_shift;
  const int begin = max(q.len - q.n, 0);                 // first position stored
  const int page_at = (begin >> c.page_shift) + int(blockIdx.x / unsigned(c.H));
  const int lo = max(begin, page_at << c.page_shift), hi = min(q.len, (page_at + 1) << c.page_shift);
  if (q.n == 0 || lo >= hi) return;
  const int page = c.table[int64_t(b) * c.width + page_at];
  if (page < 0 || page >= c.num_pages) return;
  // row of position p: first + p - (len - n)
  const int64_t from = (int64_t(q.first) + lo - (q.len - q.n)) * c.kv_stride + int64_t(head) * D;
  const int64_t codes = (int64_t(page) * c.H + head) * (int64_t(P) * D), at = int64_t(page) * c.H + head;
  if (blockIdx.z)
    append_page<FMT, D, THREADS, true>(static_cast<const uint16_t*>(c.v) + from, c.kv_stride, static_cast<uint8_t*>(c.v_pages) + codes, c.v_scales + at,
                                       c.page_shift, lo & (P - 1), hi - lo);
  else
    append_page<FMT, D, THREADS, false>(static_cast<const uint16_t*>(c.k) + from, c.kv_stride, static_cast<uint8_t*>(c.k_pages) + codes, c.k_scales + at,
                                        c.page_shift, lo & (P - 1), hi - lo);
}

template <int FMT, int D>
hipError_t go(const KvCall& c, hipStream_t s) {
  const int64_t pages = ((int64_t(c.max_new) + (1 << c.page_shift) - 2) >> c.page_shift) + 1;   // at most, of a sequence
  const dim3 grid(unsigned(pages * c.H), unsigned(c.B), 2u);
  if (c.max_new <= kFewTokens) hipLaunchKernelGGL((kv_append_kernel<FMT, D, 64>), grid, dim3(64), 0, s, c);
  else hipLaunchKernelGGL((kv_append_kernel<FMT, D, 256>), grid, dim3(256), 0, s, c);
  return hipGetLastError();
}

template <int D>
hipError_t pick(const KvCall& c, hipStream_t s) {
  return c.fmt == HQ_KV_INT8 ? go<HQ_KV_INT8, D>(c, s) : go<HQ_KV_FP8_E4M3, D>(c, s);
}

}  // namespace

hipError_t launch_kv_append(const KvCall& c, hipStream_t s) {
  switch (c.D) {
    case 64: return pick<64>(c, s);
    case 96: return pick<96>(c, s);
    case 128: return pick<128>(c, s);
    case 192: return pick<192>(c, s);
    default: return pick<256>(c, s);
  }
}

}  // namespace hq
