// attention_tile.hip -- attention over the paged 8-bit cache for many rows: prompts, pieces of prompts, many query heads to a
// head of the cache.
//
// What bounds it is arithmetic: two products of 4 D operations a (row, position), 2^x, maxima and conversions beside them. A
// workgroup takes 128 rows of one head of the cache of one sequence, 32 for each of its four waves, and all waves walk
// the same blocks of 64 positions. A block's codes are asked for from memory while the block before is worked on, converted
// once by the whole workgroup (keys to bf16, values to fp16), and handed to the waves through two LDS buffers in turn, so
// that there is one barrier a block. Products, lane layout and softmax are those of the few-row kernel.
//
// Bank conflicts: gfx950 serves a 16-byte LDS read of a wave 16 lanes at a time, eight of one lane group and the other
// eight of the next (lanes 0-3, 12-15 and 20-27; 4-11, 16-19 and 28-31; and so the upper half). Rows are stored with
// their 16-byte chunks exchanged by a key that sends these sixteen to sixteen different bank groups.
#include <hip/hip_runtime.h>

#include "attention_ops.h"

namespace hq {

namespace {

constexpr int kWaves = 4;
constexpr int kNQ = 2;
constexpr int kTileRows = 16 * kNQ * kWaves;

// LDS writes of all waves before, LDS reads after; loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Byte of chunk s of lane group q (a quarter of the channels, D / 32 chunks) of key row `row`. The chunks of a row: keys of the
// row's eight lanes of one group and of the other eight are two sets that the difference between the groups' chunks maps to
// themselves. Head sizes that are no power of two: a plane for each group, of rows an odd number of chunks long.
template <int D>
__device__ __forceinline__ int key_at(int row, int q, int s) {
  const int c = q * (D / 32) + s;
  if constexpr (D == 64) return row * 128 + ((c ^ (((row >> 1) + 2) & 7)) << 4);
  else if constexpr (D == 128) return row * 256 + ((c ^ ((row + 4) & 15)) << 4);
  else if constexpr (D == 256) return row * 512 + ((c ^ ((row & 15) ^ ((row & 8) >> 1))) << 4);
  else return ((q * kBlock + row) * (D / 32 | 1) + s) << 4;
}
// Byte of half u of the 16 positions of lane group q of channel d.
__device__ __forceinline__ int value_at(int d, int q, int u) { return d * 128 + (((2 * q + u) ^ (((d >> 1) + 2) & 7)) << 4); }

template <int D, int FMT>
__global__ __launch_bounds__(kWaves * 64, D <= 128 ? 2 : 1) void attention_tile_kernel(KvCall c) {
  constexpr int kSteps = D / 32, kTiles = D / 16;
  constexpr int kKeys = (D & (D - 1)) == 0 ? kBlock * D * 2 : 4 * kBlock * (D / 32 | 1) * 16;
  constexpr int kBuffer = kKeys + D * kBlock * 2;
  constexpr int kPieces = (D * 4 + kWaves * 64 - 1) / (kWaves * 64);    // 16-byte pieces of values a thread stages
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kBuffer];
  const int b = blockIdx.y;
  const KvSeq sq = attention_sequence(c, b);
  const int head = int(blockIdx.x % unsigned(c.H)), part = int(blockIdx.x / unsigned(c.H) % unsigned(c.n_split));
  const int rows = sq.n * c.G, tiles = (rows + kTileRows - 1) / kTileRows;
  // a sequence's last tiles, which see most, first
  const int r0 = (tiles - 1 - int(blockIdx.x / unsigned(c.H) / unsigned(c.n_split))) * kTileRows;
  if (r0 < 0) return;
  const Share sh = share_of(c, sq, r0, kTileRows);
  if (part >= sh.parts) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, col = lane & 15, quarter = lane >> 4;
  const int shift = c.page_shift, P = 1 << shift;
  const int before = sq.len - sq.n;
  const int end = min(sh.first + (part + 1) * sh.each, sh.end);
  const int32_t* table = c.table + int64_t(b) * c.width;

  // Staging: a thread takes a quarter of one key's channels (the 16 keys of a wave are of one page), and 16-byte pieces of
  // values (channel, 16 positions). Pages are asked for two blocks ahead, codes and scales one.
  const int key = tid >> 2, piece = tid & 3;
  const int key_row = 16 * ((key >> 2) & 3) + 4 * (key >> 4) + (key & 3);
  int spage, vpage;        // of this lane's positions, and of its piece of values
  uint2 kc[kSteps];
  u32x4 vc[kPieces];
  int live;                // positions of this thread's values that exist
  float ks, vs;            // scales of this lane's positions
  bool there;
  const auto load_pages = [&](int blk) {
    const int sg = blk * kBlock + 16 * quarter, vg = blk * kBlock + 16 * piece;
    const int most = sq.len - 1;
    spage = table[min(sg, most) >> shift];      // (of the last page where there is none: not used)
    vpage = table[min(vg, most) >> shift];
  };
  const uint8_t* const kp = static_cast<const uint8_t*>(c.k_pages) + ((int64_t(head) << shift) + (key & 15)) * D + piece * (D / 4);
  const uint8_t* const vp = static_cast<const uint8_t*>(c.v_pages) + ((int64_t(head) * D + (tid >> 2)) << shift);
  const auto load = [&](int blk) {
    const int base = blk * kBlock;
    const int kg = base + 16 * wave, vg = base + 16 * piece, sg = base + 16 * quarter;
    there = sg < sq.len && spage >= 0 && spage < c.num_pages;
    const bool vthere = vg < sq.len && vpage >= 0 && vpage < c.num_pages;
    live = vthere ? sq.len - vg : 0;
    const uint32_t page = there ? spage : 0, from = vthere ? vpage : 0;
    const uint32_t kpage = __builtin_amdgcn_readlane(page, 16 * wave);
    const uint8_t* k = kp + uint64_t(kpage) * c.page_bytes + (kg & (P - 1)) * D;
    const uint8_t* v = vp + uint64_t(from) * c.page_bytes + (vg & (P - 1));
#pragma unroll
    for (int s = 0; s < kSteps; ++s) kc[s] = *reinterpret_cast<const uint2*>(k + 8 * s);
#pragma unroll
    for (int e = 0; e < kPieces; ++e)
      if (D % 64 == 0 || (tid >> 2) + 64 * e < D) vc[e] = ldg16(v + (int64_t(64 * e) << shift));
    const uint64_t at = uint64_t(page) * unsigned(c.H) + unsigned(head);
    ks = c.k_scales[at];
    vs = c.v_scales[at];
  };
  const auto store = [&](uint8_t* to) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) *reinterpret_cast<bf16x8*>(to + key_at<D>(key_row, piece, s)) = codes_bf16<FMT>(kc[s].x, kc[s].y);
    if (__any(live < 16)) {
#pragma unroll
      for (int e = 0; e < kPieces; ++e) vc[e] = live_codes(vc[e], live);
    }
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const int d = (tid >> 2) + 64 * e;
      if (D % 64 != 0 && d >= D) break;
      *reinterpret_cast<f16x8*>(to + kKeys + value_at(d, piece, 0)) = codes_f16<FMT>(vc[e][0], vc[e][1]);
      *reinterpret_cast<f16x8*>(to + kKeys + value_at(d, piece, 1)) = codes_f16<FMT>(vc[e][2], vc[e][3]);
    }
  };
  int blk = sh.first + part * sh.each;
  if (blk < end) {
    load_pages(blk);
    load(blk);
    load_pages(blk + 1);
  }

  bf16x8 qf[kNQ][kSteps];
  int pos[kNQ];
  const int w0 = r0 + wave * 16 * kNQ;      // the wave's first row
#pragma unroll
  for (int n = 0; n < kNQ; ++n) {
    const int r = w0 + 16 * n + col;
    const int i = r / c.G, g = r - i * c.G;
    pos[n] = r < rows ? before + i : -1;
    const auto* qp = static_cast<const uint16_t*>(c.q) + (int64_t(sq.first) + i) * c.q_stride + int64_t(head * c.G + g) * D + quarter * (D / 4);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) qf[n][s] = r < rows ? query8(qp + 8 * s, c.q_sign) : bf16x8{};
  }
  const int pos_first = before + w0 / c.G;
  const int pos_last = w0 < rows ? before + (min(w0 + 16 * kNQ, rows) - 1) / c.G : -1;

  Rows<kNQ, kTiles> st;
  st.clear();
  for (int buffer = 0; blk < end; ++blk, buffer ^= 1) {
    uint8_t* at = lds + buffer * kBuffer;
    store(at);
    float f = ks * c.scale_log2;
    const float lv = there ? log2f(vs) : -INFINITY;
    const bool here = there;
    if (blk + 1 < end) {
      load(blk + 1);
      load_pages(blk + 2);
    }
    lds_barrier();
    const int base = blk * kBlock, vg = base + 16 * quarter;
    // blocks that none of the wave's rows sees
    if (base > pos_last || (c.window > 0 && base + kBlock - 1 <= pos_first - c.window)) continue;
    f32x4 score[kNQ][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int n = 0; n < kNQ; ++n) score[n][i] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(at + key_at<D>(16 * i + col, quarter, s));
#pragma unroll
        for (int n = 0; n < kNQ; ++n) score[n][i] = mfma_bf16(kf, qf[n][s], score[n][i]);
      }
    }
    if (base + kBlock - 1 > pos_first || (c.window > 0 && base <= pos_last - c.window) || __any(!here)) {
      mask_scores<kNQ>(score, pos, vg, c.window, here, f);
      f = 1.0f;
    }
    f16x8 weight[kNQ][2];
    st.step(score, f, lv, weight);
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f16x8 vf = *reinterpret_cast<const f16x8*>(at + kKeys + value_at(16 * t + col, quarter, u));
#pragma unroll
        for (int n = 0; n < kNQ; ++n) st.acc[n][t] = mfma_f16(vf, weight[n][u], st.acc[n][t]);
      }
  }

#pragma unroll
  for (int n = 0; n < kNQ; ++n) {
    const int r = w0 + 16 * n + col;
    const float total = row_sum(st.sum[n]), unit = st.unit(n);
    if (r >= rows) continue;
    const int i = r / c.G, h = head * c.G + r % c.G;
    if (sh.parts == 1) {
      const float inv = total == 0.0f ? 0.0f : unit / total;
      auto* out = static_cast<uint16_t*>(c.out) + ((int64_t(sq.first) + i) * c.Hq + h) * D + 4 * quarter;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const f32x4& o = st.acc[n][t];
        *reinterpret_cast<uint2*>(out + 16 * t) = make_uint2(f32x2_to_bf16x2_rne(o[0] * inv, o[1] * inv), f32x2_to_bf16x2_rne(o[2] * inv, o[3] * inv));
      }
    } else {
      const int64_t to = part_row(c, sq, b, i, h) + part;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        f32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = st.acc[n][t][j] * unit;
        *reinterpret_cast<f32x4*>(c.ws_o + to * D + 16 * t + 4 * quarter) = o;
      }
      if (quarter == 0) *reinterpret_cast<float2*>(c.ws_ml + 2 * to) = make_float2(st.top[n], total);
    }
  }
}

template <int D>
hipError_t go(const KvCall& c, hipStream_t s) {
  const int64_t rows = int64_t(c.hi_n) * c.G;
  const dim3 grid(unsigned((rows + kTileRows - 1) / kTileRows) * unsigned(c.n_split) * unsigned(c.H), unsigned(c.B));
  if (c.fmt == HQ_KV_INT8) hipLaunchKernelGGL((attention_tile_kernel<D, HQ_KV_INT8>), grid, dim3(kWaves * 64), 0, s, c);
  else hipLaunchKernelGGL((attention_tile_kernel<D, HQ_KV_FP8_E4M3>), grid, dim3(kWaves * 64), 0, s, c);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_tiles(const KvCall& c, hipStream_t s) {
  switch (c.D) {
    case 64: return go<64>(c, s);
    case 96: return go<96>(c, s);
    case 128: return go<128>(c, s);
    case 192: return go<192>(c, s);
    default: return go<256>(c, s);
  }
}

}  // namespace hq
