// attention_ops.h -- what the two attention kernels share: the lane layout of a block's scores, the running
// softmax of its rows, and how a sequence's positions are shared out.
//
// A wave works on NQ tiles of 16 rows (query tokens times the heads that share a head of the cache) and blocks of 64
// positions. In every product a row is a matrix column: lane l holds, for row l % 16 of each tile, the 16 scores of
// positions 16 (l / 16) .. + 15 of the block (element r of vector i: position 4 i + r of those). 16 positions never
// cross a page, so a lane has one scale of K, a factor of its scores, and one of V, a factor of its weights. The scores
// leave the first product as the second one takes them: nothing is exchanged between lanes but the row's maxima.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_ops.h"
#include "internal.h"
#include "kv_cache.h"

namespace hq {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 64;   // positions of a block

// Eight codes as bf16 (keys, beside the queries) or as fp16 (values): exact in both.
template <int FMT>
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t lo, uint32_t hi) {
  if constexpr (FMT == HQ_KV_INT8) return dequant_int8x8(lo, hi);
  else return dequant_fp8x8(lo, hi);
}

template <int FMT>
__device__ __forceinline__ f16x8 codes_f16(uint32_t lo, uint32_t hi) {
  if constexpr (FMT == HQ_KV_INT8) {
    // 0x6400 | u is 1024 + u in fp16; u = code + 128
    const auto two = [](uint32_t u, uint32_t sel) {
      return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, sel)) - f16x2{_Float16(1152), _Float16(1152)};
    };
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    const f16x2 a = two(lo, 0x04010400u), b = two(lo, 0x04030402u), c = two(hi, 0x04010400u), d = two(hi, 0x04030402u);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
}

__device__ __forceinline__ f32x4 mfma_f16(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }   // results below 2^-126 are 0

// Maximum and sum over the four lanes that hold one row (lanes l, l ^ 16, l ^ 32, l ^ 48).
template <class F>
__device__ __forceinline__ float over_quarters(float v, F join) {
  auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = join(__uint_as_float(p[0]), __uint_as_float(p[1]));
  p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return join(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float row_max(float v) {
  return over_quarters(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float row_sum(float v) {
  return over_quarters(v, [](float a, float b) { return a + b; });
}

// Running softmax of the rows a lane holds. With x = sm_scale * log2(e) * q . k and s_v the scale of the position's values:
//   sum = sum 2^(x - top)  (this lane's positions),   acc = sum 2^(x + log2 s_v - top - rel) * code,
// with references top, below the maximum of x seen so far, and top + rel, kRaise below that of x + log2 s_v, by little enough that a
// lane's 16 terms add up to kMost, and its 16 weights to kMostWeights, at most: the sums that are made anyhow tell, so that the maxima
// are taken, over a row's four lanes, and what was summed before is brought to new references, only in blocks where one has to move
// (the first and a few others).
// The second reference is kept from the first: scores may be of any size, also one at which log2 s_v is lost beside them.
// The weights 2^(x + log2 s_v - top - rel) enter the product with the codes as fp16: each is off by 2^-11 of itself or 2^-35 of the
// row's largest, whatever the scales (a bf16 weight, off by 2^-8, made the result's error half as large again as the
// rounding of the result itself). Statistics and sums are fp32. The largest is between 2^kRaise and fp16's end, so that nearly all of
// fp16's range is below it: in a row whose first token takes 0.999 of the weight, with a value of 0, the others have 2^-25 of it. Error of
// such rows in units of the result's own rounding, on 20000 or 30000 positions, and time of 4 prompts of 4500, where a raised
// reference moves more often: kRaise 0 (and weights to 2^8) up to 377, 467 us; 8 1.69, 468; 10 1.21, 469; 11 1.19, 488.
constexpr float kMost = 256.0f;     // 2^kSlack
constexpr float kSlack = 8.0f;
constexpr float kRaise = 10.0f;
constexpr float kLower = 0x1p-10f;  // 2^-kRaise
constexpr float kMostWeights = 65504.0f;      // the largest fp16
constexpr float kFar = -60.0f;
constexpr float kLarge = 4096.0f;   // (below, a fused product is within 2^-12 of the rounded one)
constexpr float kNone = -3e38f;     // top of a row that has seen nothing: its scores are -infinity, its sums 0
constexpr float kLeast = -1e37f;    // rel of a row that has seen no value but 0: lv - rel - top stays finite whatever the scores are

template <int NQ, int TILES>
struct Rows {
  f32x4 acc[NQ][TILES];
  float top[NQ], rel[NQ], sum[NQ];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      top[n] = kNone;
      rel[n] = sum[n] = 0.0f;
#pragma unroll
      for (int t = 0; t < TILES; ++t) acc[n][t] = f32x4{0, 0, 0, 0};
    }
  }

  // A block's scores to weights. Scores are products of q and k codes, ks >= 0 makes them x (where masked they are -infinity or
  // x already, and ks is 1); lv = log2 of the values' scale, -infinity where that is 0 or there is no page.
  // The weights are made with the references there are, and again where those move.
  __device__ __forceinline__ void step(f32x4 (&score)[NQ][4], float ks, float lv, f16x8 (&weight)[NQ][2]) {
    float part[NQ], more[NQ], e[NQ];      // e: log2 of the weights' unit to that of the sum's terms
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      e[n] = lv - rel[n];
      weigh(score[n], ks, e[n] - top[n], e[n], weight[n], part[n], more[n]);
    }
    settle(weight);
    bool rare = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) rare |= !(part[n] <= kMostWeights && more[n] <= kMost && e[n] > kFar);
    if (__any(rare)) {
#pragma clang fp contract(off)
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        // new references; a row goes by its own sums: what the tile's other rows hold does not change its bits
        const float m = block_max(score[n]) * ks, rm = row_max(m);
        // (a lane whose weights vanish beside its part of the sum: by its maximum)
        const bool far_now = !(e[n] > kFar);
        const bool moves = row_max((far_now ? m > top[n] + kSlack : !(part[n] <= kMostWeights && more[n] <= kMost)) ? 1.0f : 0.0f) > 0.0f;
        const float top1 = moves ? fmaxf(top[n], rm) : top[n];
        const float old = fmaxf(rel[n] + (top[n] - top1), kLeast), rw = row_max((m - top1) + lv) - kRaise;
        const float rel1 = moves ? fmaxf(old, rw) : rel[n];
        if (__any(moves && top[n] > kNone)) {      // (where a row had seen nothing, sum and acc are 0)
          sum[n] *= exp2_fast(top[n] - top1);
          const float shrink = exp2_fast(old - rel1);
#pragma unroll
          for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[n][t][r] *= shrink;
        }
        top[n] = top1;
        rel[n] = rel1;
        e[n] = lv - rel1;
        // Large scores go by their products' distances from the new reference, rounded before: 0 for the one that set it, where the
        // fused form leaves the rounding of the reference (2^40 for scores of 2^64).
        const bool large = moves && !(fabsf(top1) < kLarge);
        const float unit = large ? 1.0f : ks, from = large ? 0.0f : -top1;
        if (__any(large)) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float x = score[n][k >> 2][k & 3];
            score[n][k >> 2][k & 3] = large ? x * ks - top1 : x;
          }
        }
        // Scales so far apart (or 0) that a weight vanishes where its part of the sum does not: that part by itself.
        const bool far = !(e[n] > kFar);
        if (__any(far)) {
          float s = 0.0f;
          const float at = top1 > kNone ? from : 0.0f;
#pragma unroll
          for (int k = 0; k < 16; ++k) s += exp2_fast(fmaf(score[n][k >> 2][k & 3], unit, at));
          sum[n] += far ? s : 0.0f;
        }
        weigh(score[n], unit, e[n] + from, e[n], weight[n], part[n], more[n]);
      }
      settle(weight);
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) sum[n] += e[n] > kFar ? more[n] : 0.0f;
  }

  static __device__ __forceinline__ float block_max(const f32x4 (&x)[4]) {
    const auto four = [](const f32x4& v) { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); };
    return fmaxf(fmaxf(four(x[0]), four(x[1])), fmaxf(four(x[2]), four(x[3])));
  }

  // Weights 2^(score * ks + start), their sum over the lane's positions, and that of 2^(x - top), which is 2^-e times the first.
  static __device__ __forceinline__ void weigh(const f32x4 (&score)[4], float ks, float start, float e, f16x8 (&weight)[2], float& part, float& more) {
    float four[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float p[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) p[r] = exp2_fast(fmaf(score[i][r], ks, start));
      four[i] = (p[0] + p[1]) + (p[2] + p[3]);
      u32x4 w = __builtin_bit_cast(u32x4, weight[i >> 1]);
#pragma unroll
      for (int r = 0; r < 4; r += 2) {
        const f32x2 two = {p[r], p[r + 1]};
        w[2 * (i & 1) + r / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, f16x2));
      }
      weight[i >> 1] = __builtin_bit_cast(f16x8, w);
    }
    part = (four[0] + four[1]) + (four[2] + four[3]);
    more = part * exp2_fast(-e);
  }

  // (weights made here, not behind the branch that may make them again)
  static __device__ __forceinline__ void settle(f16x8 (&weight)[NQ][2]) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      u32x4 u = __builtin_bit_cast(u32x4, weight[n][0]), v = __builtin_bit_cast(u32x4, weight[n][1]);
      asm volatile("" : "+v"(u), "+v"(v));
      weight[n][0] = __builtin_bit_cast(f16x8, u);
      weight[n][1] = __builtin_bit_cast(f16x8, v);
    }
  }
};

// Parts hand on averages, not sums: a sum of values near the largest bf16 leaves fp32's range where their average does not. They
// are kept as a quarter, since a code rounded up and its scale may be twice that bf16; the join gives each its share of the total, which
// is 1 at most, times 4. 0 for rows that have seen nothing.
constexpr float kKept = 0.25f;
__device__ __forceinline__ float inverse(float total) { return total == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(total); }   // (off by 2^-23 at most)
// acc * lowered(sum) * unit(rel) is the average of what a row has seen: two factors, which may each be far from 1.
__device__ __forceinline__ float lowered(float total) { return inverse(total) * kLower; }
__device__ __forceinline__ float unit(float rel) { return exp2f(rel + kRaise); }

// Scores of positions that row `pos` (a position) does not see become -infinity, the others x. vg: the lane's first position.
template <int NQ>
__device__ __forceinline__ void mask_scores(f32x4 (&score)[NQ][4], const int (&pos)[NQ], int vg, int window, bool there, float ks) {
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int t = vg + e;
      const bool seen = there && t <= pos[n] && (window == 0 || t > pos[n] - window);
      score[n][e >> 2][e & 3] = seen ? score[n][e >> 2][e & 3] * ks : -INFINITY;
    }
}

// 16 codes of values (positions vg ..) with those behind the sequence's end, which are whatever the page holds, made 0: a NaN
// there times a weight of 0 is NaN.
__device__ __forceinline__ u32x4 live_codes(u32x4 v, int live) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int left = live - 4 * w;
    v[w] &= left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
  }
  return v;
}

// The blocks that the rows [r0, r0 + rows) of a sequence see, and how they are shared out: part s takes the blocks
// first + s * each .. The join reads the same numbers.
struct Share {
  int first, end, each, parts;
};

__device__ __forceinline__ Share share_of(const KvCall& c, const KvSeq& q, int r0, int rows) {
  const int last = min(r0 + rows, q.n * c.G) - 1;
  const int hi = q.len - q.n + last / c.G;                    // position of the last row
  const int lo = q.len - q.n + r0 / c.G - c.window + 1;       // first position that the first row sees
  Share s;
  s.first = c.window > 0 ? max(lo, 0) / kBlock : 0;
  s.end = hi < 0 ? s.first : hi / kBlock + 1;
  const int blocks = s.end - s.first;
  s.each = max(c.each, (blocks + c.n_split - 1) / c.n_split);
  s.parts = max((blocks + s.each - 1) / s.each, 1);
  return s;
}

// Where the partial results of (token i of sequence b, query head) begin, in rows of n_split parts.
__device__ __forceinline__ int64_t part_row(const KvCall& c, const KvSeq& q, int b, int i, int head) {
  const int64_t token = c.by_token ? int64_t(q.first) + i : int64_t(b) * c.hi_n + i;
  return (token * c.Hq + head) * c.n_split;
}

// The sequences of this launch: those with lo_n .. hi_n new tokens.
__device__ __forceinline__ KvSeq attention_sequence(const KvCall& c, int b) {
  KvSeq q = kv_sequence(c, b);
  if (q.n < c.lo_n || q.n > c.hi_n) q.n = 0;
  return q;
}

// A lane's part of its query rows, r0 + 16 n + l % 16: a quarter of the channels each. Rows past the last one hold that one, so that
// the loads are in flight together, not each in a branch of its own; nothing of them is written.
template <int NQ, int STEPS>
__device__ __forceinline__ void load_queries(const KvCall& c, const KvSeq& sq, int head, int r0, int rows, bf16x8 (&q)[NQ][STEPS]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = min(r0 + 16 * n + (lane & 15), rows - 1), i = r / c.G, g = r - i * c.G;
    const auto* p = static_cast<const uint16_t*>(c.q) + (int64_t(sq.first) + i) * c.q_stride + int64_t(head * c.G + g) * (32 * STEPS) + (lane >> 4) * (8 * STEPS);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) q[n][s] = __builtin_bit_cast(bf16x8, ldg16(p + 8 * s));
  }
}
// Negated where sm_scale is negative (its size alone is a factor of the keys' scale).
template <int NQ, int STEPS>
__device__ __forceinline__ void sign_queries(const KvCall& c, bf16x8 (&q)[NQ][STEPS]) {
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      u32x4 x = __builtin_bit_cast(u32x4, q[n][s]);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] ^= c.q_sign;
      q[n][s] = __builtin_bit_cast(bf16x8, x);
    }
}

}  // namespace hq
