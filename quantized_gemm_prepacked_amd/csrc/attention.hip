// attention.hip -- attention over the paged 8-bit cache: softmax(sm_scale * q . k) v with the running
// maximum and sum of each row, one pass over the keys and values.
//
// The rows of a (sequence, head of the cache) are its n query tokens times the G query heads that share
// the head: row r is token r / G, head r % G, so that keys and values are read once for all of them. A workgroup takes
// 16 * NQ rows and a range of the positions; its four waves take blocks of 64 positions in turn and join
// their results through LDS. Few rows and a long past: the positions are split over workgroups as well, and
// a second launch joins the parts.
//
// Products of a block, by 16x16x32 matrix instructions without a pass through LDS:
//   S^T = K . Q^T    tile i of 4: A row m is position 16 (m / 4) + 4 i + (m % 4) of the block, so that lane l
//                    ends up with the 16 scores of positions 16 (l / 16) .. + 15 for row l % 16;
//   O^T += V^T . P^T A row m is channel 16 t + m, whose 16 codes of the lane group's positions are one 16-byte load
//                    from the transposed page; P^T is what the lane already holds.
// 16 positions never cross a page, so a lane group has one page, one scale of K (a factor of its scores) and one of V
// (a factor of its probabilities). Channel order inside a dot product is free: a lane group takes a quarter of them.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device_ops.h"
#include "internal.h"
#include "kv_cache.h"

namespace hq {

namespace {

constexpr int kWaves = 4;
constexpr int kBlock = 64;   // positions of a block

template <int FMT>
__device__ __forceinline__ bf16x8 dequant8(uint32_t lo, uint32_t hi) {
  if constexpr (FMT == HQ_KV_INT8) return dequant_int8x8(lo, hi);
  else return dequant_fp8x8(lo, hi);
}

// The blocks of 64 positions that the rows [r0, r0 + rows) of a sequence see, and how they are shared out:
// part s takes blocks first + s * each .. The join reads the same numbers.
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
  s.each = max((blocks + c.n_split - 1) / c.n_split, kWaves);
  s.parts = max((blocks + s.each - 1) / s.each, 1);
  return s;
}

// Where the partial results of (token i of sequence b, head) begin, in rows of n_split parts.
__device__ __forceinline__ int64_t part_row(const KvCall& c, const KvSeq& q, int b, int i, int head) {
  const int64_t token = c.by_token ? int64_t(q.first) + i : int64_t(b) * c.max_new + i;
  return (token * c.Hq + head) * c.n_split;
}

template <int D, int FMT, int NQ>
__global__ __launch_bounds__(kWaves * 64) void attention_kernel(KvCall c) {
  constexpr int kSteps = D / 32;      // matrix instructions of a dot product
  constexpr int kTiles = D / 16;      // 16-channel tiles of the output
  constexpr int kRows = 16 * NQ;
  const int b = blockIdx.y;
  const KvSeq sq = kv_sequence(c, b);
  // heads next to each other, so that with eight of them a head's workgroups run on one XCD and share its L2
  const int head = int(blockIdx.x % unsigned(c.H));
  const int part = int(blockIdx.x / unsigned(c.H) % unsigned(c.n_split));
  const int r0 = int(blockIdx.x / unsigned(c.H) / unsigned(c.n_split)) * kRows;
  const int rows = sq.n * c.G;
  if (r0 >= rows) return;
  const Share sh = share_of(c, sq, r0, kRows);
  if (part >= sh.parts) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, col = lane & 15, quarter = lane >> 4;
  const int shift = c.page_shift, P = 1 << shift;
  const int before = sq.len - sq.n;

  // this lane's rows, one of each 16: query fragments and the last position seen
  bf16x8 qf[NQ][kSteps];
  int pos[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = r0 + 16 * n + col;
    const int i = r / c.G, g = r - i * c.G;
    pos[n] = r < rows ? before + i : -1;
    const auto* qp = static_cast<const __bf16*>(c.q) + (int64_t(sq.first) + i) * c.q_stride + int64_t(head * c.G + g) * D + quarter * (D / 4);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (r < rows) qf[n][s] = *reinterpret_cast<const bf16x8*>(qp + 8 * s);
      else qf[n][s] = bf16x8{};
    }
  }
  const int pos_first = before + r0 / c.G;                        // of the first row, and of the last one
  const int pos_last = before + (min(r0 + kRows, rows) - 1) / c.G;

  f32x4 acc[NQ][kTiles];
  float top[NQ], sum[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    top[n] = -INFINITY;
    sum[n] = 0.0f;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[n][t] = f32x4{0, 0, 0, 0};
  }

  const auto* kp = static_cast<const uint8_t*>(c.k_pages);
  const auto* vp = static_cast<const uint8_t*>(c.v_pages);
  const int32_t* table = c.table + int64_t(b) * c.width;
  const int end = min(sh.first + (part + 1) * sh.each, sh.end);
  for (int blk = sh.first + part * sh.each + wave; blk < end; blk += kWaves) {
    const int base = blk * kBlock;
    // pages of the 16 positions whose keys this lane loads (its A rows) and whose values it holds
    const int kg = base + 16 * (col >> 2), vg = base + 16 * quarter;
    int kpage = kg < sq.len ? table[kg >> shift] : -1, vpage = vg < sq.len ? table[vg >> shift] : -1;
    const bool there = vpage >= 0 && vpage < c.num_pages;
    if (kpage < 0 || kpage >= c.num_pages) kpage = 0;
    if (!there) vpage = 0;
    const uint8_t* kb = kp + ((int64_t(kpage) * c.H + head) * P + (kg & (P - 1)) + (col & 3)) * D + quarter * (D / 4);
    const uint8_t* vb = vp + ((int64_t(vpage) * c.H + head) * D + col) * P + (vg & (P - 1));
    uint2 kc[4][kSteps];
    u32x4 vc[kTiles];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) kc[i][s] = *reinterpret_cast<const uint2*>(kb + 4 * i * D + 8 * s);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) vc[t] = ldg16(vb + int64_t(16 * t) * P);
    // (a page that does not exist stands for page 0, whose scale may be anything: a NaN times a probability of 0 is NaN)
    const float ks = c.k_scales[int64_t(vpage) * c.H + head] * c.scale_log2, vs = there ? c.v_scales[int64_t(vpage) * c.H + head] : 0.0f;

    f32x4 score[NQ][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) score[n][i] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const bf16x8 kf = dequant8<FMT>(kc[i][s].x, kc[i][s].y);
#pragma unroll
        for (int n = 0; n < NQ; ++n) score[n][i] = mfma_bf16(kf, qf[n][s], score[n][i]);
      }
    }
    const bool edge = base + kBlock - 1 > pos_first || (c.window > 0 && base <= pos_last - c.window) || __any(!there);
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          score[n][i][r] *= ks;
          if (edge) {
            const int t = vg + 4 * i + r;
            if (!there || t > pos[n] || (c.window > 0 && t <= pos[n] - c.window)) score[n][i][r] = -INFINITY;
          }
        }
    // codes behind the sequence's end are whatever the page holds: a NaN there times a probability of 0 is NaN
    if (edge) {
      const int live = there ? min(max(sq.len - vg, 0), 16) : 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int left = live - 4 * w;
        const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) vc[t][w] &= keep;
      }
    }

    bf16x8 pf[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float m = top[n];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, score[n][i][r]);
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      const float ref = m == -INFINITY ? 0.0f : m;      // a row that has seen nothing yet
      const float old = exp2f(top[n] - ref);
      top[n] = m;
      if (__any(old != 1.0f)) {
        sum[n] *= old;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[n][t][r] *= old;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] = exp2f(score[n][2 * u + (j >> 2)][j & 3] - ref);
          sum[n] += p[j];
        }
        const u32x4 w = {f32x2_to_bf16x2_rne(p[0] * vs, p[1] * vs), f32x2_to_bf16x2_rne(p[2] * vs, p[3] * vs),
                         f32x2_to_bf16x2_rne(p[4] * vs, p[5] * vs), f32x2_to_bf16x2_rne(p[6] * vs, p[7] * vs)};
        pf[n][u] = __builtin_bit_cast(bf16x8, w);
      }
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bf16x8 vf = dequant8<FMT>(vc[t][2 * u], vc[t][2 * u + 1]);
#pragma unroll
        for (int n = 0; n < NQ; ++n) acc[n][t] = mfma_bf16(vf, pf[n][u], acc[n][t]);
      }
  }

  // the four waves' parts, joined 16 rows at a time
  __shared__ float tops[kWaves][16], sums[kWaves][16];
  __shared__ float parts[kWaves][16][D + 4];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float l = sum[n];
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (n) __syncthreads();
    if (quarter == 0) {
      tops[wave][col] = top[n];
      sums[wave][col] = l;
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) *reinterpret_cast<f32x4*>(&parts[wave][col][16 * t + 4 * quarter]) = acc[n][t];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * (D / 4); e += kWaves * 64) {
      const int row = e / (D / 4), d = (e % (D / 4)) * 4;
      const int r = r0 + 16 * n + row;
      if (r >= rows) continue;
      float m = tops[0][row];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) m = fmaxf(m, tops[w][row]);
      const float ref = m == -INFINITY ? 0.0f : m;
      float total = 0.0f;
      f32x4 o = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = exp2f(tops[w][row] - ref);
        total += f * sums[w][row];
        const f32x4 x = *reinterpret_cast<const f32x4*>(&parts[w][row][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += f * x[j];
      }
      const int i = r / c.G, h = head * c.G + r % c.G;
      if (sh.parts == 1) {
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        const uint2 w = {f32x2_to_bf16x2_rne(o[0] * inv, o[1] * inv), f32x2_to_bf16x2_rne(o[2] * inv, o[3] * inv)};
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.out) + ((int64_t(sq.first) + i) * c.Hq + h) * D + d) = w;
      } else {
        const int64_t at = part_row(c, sq, b, i, h) + part;
        *reinterpret_cast<f32x4*>(c.ws_o + at * D + d) = o;
        if (d == 0) *reinterpret_cast<float2*>(c.ws_ml + 2 * at) = make_float2(m, total);
      }
    }
  }
}

// The parts of a row joined: one wave a (token, query head).
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(KvCall c, int tile_rows) {
  const int b = blockIdx.y;
  const KvSeq sq = kv_sequence(c, b);
  const int head = int(blockIdx.x % unsigned(c.H)), r = int(blockIdx.x / unsigned(c.H)) * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (r >= sq.n * c.G) return;
  const Share sh = share_of(c, sq, r / tile_rows * tile_rows, tile_rows);
  if (sh.parts == 1) return;
  const int i = r / c.G, h = head * c.G + r % c.G;
  const int64_t at = part_row(c, sq, b, i, h);
  float m = -INFINITY;
  for (int s = 0; s < sh.parts; ++s) m = fmaxf(m, c.ws_ml[2 * (at + s)]);
  const float ref = m == -INFINITY ? 0.0f : m;
  constexpr int kEach = (D + 63) / 64;
  float o[kEach] = {}, total = 0.0f;
  for (int s = 0; s < sh.parts; ++s) {
    const float2 ml = *reinterpret_cast<const float2*>(c.ws_ml + 2 * (at + s));
    const float f = exp2f(ml.x - ref);
    total += f * ml.y;
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (lane + 64 * j < D) o[j] += f * c.ws_o[(at + s) * D + lane + 64 * j];
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
  for (int j = 0; j < kEach; ++j)
    if (lane + 64 * j < D) static_cast<uint16_t*>(c.out)[((int64_t(sq.first) + i) * c.Hq + h) * D + lane + 64 * j] = f32_to_bf16_rne(o[j] * inv);
}

constexpr int kMaxSplit = 64;

// Rows of a workgroup: two tiles of 16 where there are more than 16.
int tile_rows(const KvCall& c) { return int64_t(c.max_new) * c.G > 16 ? 32 : 16; }

template <int D, int FMT, int NQ>
hipError_t go(const KvCall& c, hipStream_t s) {
  const int64_t rows = int64_t(c.max_new) * c.G;
  const unsigned tiles = unsigned((rows + 16 * NQ - 1) / (16 * NQ));
  hipLaunchKernelGGL((attention_kernel<D, FMT, NQ>), dim3(tiles * unsigned(c.n_split) * unsigned(c.H), unsigned(c.B)), dim3(kWaves * 64), 0, s, c);
  if (c.n_split > 1)
    hipLaunchKernelGGL((attention_join_kernel<D>), dim3(unsigned((rows + 3) / 4) * unsigned(c.H), unsigned(c.B)), dim3(256), 0, s, c, 16 * NQ);
  return hipGetLastError();
}

template <int D>
hipError_t pick(const KvCall& c, hipStream_t s) {
  const bool two = tile_rows(c) == 32;
  if (c.fmt == HQ_KV_INT8) return two ? go<D, HQ_KV_INT8, 2>(c, s) : go<D, HQ_KV_INT8, 1>(c, s);
  return two ? go<D, HQ_KV_FP8_E4M3, 2>(c, s) : go<D, HQ_KV_FP8_E4M3, 1>(c, s);
}

}  // namespace

int64_t attention_groups(const KvCall& c) {
  const int64_t rows = int64_t(c.max_new) * c.G;
  return (rows + tile_rows(c) - 1) / tile_rows(c) * c.H * c.B;
}

AttentionPlan plan_attention(const KvCall& c, int64_t max_kv) {
  const int64_t groups = attention_groups(c), blocks = (max_kv + kBlock - 1) / kBlock;
  const int64_t split = std::min((1024 + groups - 1) / groups, (blocks + kWaves - 1) / kWaves);
  AttentionPlan p{};
  p.n_split = int(std::max<int64_t>(1, std::min<int64_t>(split, kMaxSplit)));
  p.by_token = c.T <= int64_t(c.B) * c.max_new;
  const int64_t slots = p.by_token ? c.T : int64_t(c.B) * c.max_new;
  if (p.n_split > 1) {
    p.ml_offset = size_t(slots) * c.Hq * p.n_split * c.D * 4;
    p.ws_bytes = p.ml_offset + size_t(slots) * c.Hq * p.n_split * 8;
  }
  return p;
}

hipError_t launch_attention(const KvCall& c, hipStream_t s) {
  switch (c.D) {
    case 64: return pick<64>(c, s);
    case 96: return pick<96>(c, s);
    case 128: return pick<128>(c, s);
    case 192: return pick<192>(c, s);
    default: return pick<256>(c, s);
  }
}

}  // namespace hq
