// attention_tile.hip -- attention over the paged 8-bit cache for many rows: prompts, pieces of prompts, many query heads to a
// head of the cache.
//
// What bounds it is arithmetic: two products of 4 D operations a (row, position), 2^x, maxima and conversions beside them. A
// workgroup takes 128 rows of one head of the cache of one sequence, 32 for each of its four waves, and all waves walk
// the same blocks of 64 positions. A block's codes are asked for from memory while the block before is worked on, converted
// once by the whole workgroup (keys to bf16, values to fp16), and handed to the waves through two LDS buffers in turn, so
// that there is one barrier a block. Products, lane layout and softmax are those of the few-row kernel.
//
// LDS rows are 16 bytes longer than their values: the sixteen rows that one read touches start in different banks.
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

template <int D, int FMT>
__global__ __launch_bounds__(kWaves * 64, D <= 128 ? 2 : 1) void attention_tile_kernel(KvCall c) {
  constexpr int kSteps = D / 32, kTiles = D / 16;
  constexpr int kKeyRow = 2 * D + 16, kValueRow = 2 * kBlock + 16;      // bytes of an LDS row
  constexpr int kKeys = kBlock * kKeyRow, kBuffer = kKeys + D * kValueRow;
  constexpr int kPieces = (D * 4 + kWaves * 64 - 1) / (kWaves * 64);    // 16-byte pieces of values a thread stages
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][kBuffer];
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

  // Staging: a thread takes a quarter of one key's channels, and 16-byte pieces of values (channel, 16 positions).
  const int key = tid >> 2, piece = tid & 3;
  const int key_row = 16 * ((key >> 2) & 3) + 4 * (key >> 4) + (key & 3);
  uint2 kc[kSteps];
  u32x4 vc[kPieces];
  int live;                // positions of this thread's values that exist
  float ks, vs;            // scales of this lane's positions
  bool there;
  const auto load = [&](int blk) {
    const int base = blk * kBlock;
    const int kg = base + key, vg = base + 16 * piece, sg = base + 16 * quarter;
    int kpage = kg < sq.len ? table[kg >> shift] : -1, vpage = vg < sq.len ? table[vg >> shift] : -1, spage = sg < sq.len ? table[sg >> shift] : -1;
    if (kpage < 0 || kpage >= c.num_pages) kpage = 0;
    live = vpage >= 0 && vpage < c.num_pages ? sq.len - vg : 0;
    if (live == 0) vpage = 0;
    there = spage >= 0 && spage < c.num_pages;
    if (!there) spage = 0;
    const uint8_t* kp = static_cast<const uint8_t*>(c.k_pages) + ((int64_t(kpage) * c.H + head) * P + (kg & (P - 1))) * D + piece * (D / 4);
    const uint8_t* vp = static_cast<const uint8_t*>(c.v_pages) + (int64_t(vpage) * c.H + head) * D * P + (vg & (P - 1));
#pragma unroll
    for (int s = 0; s < kSteps; ++s) kc[s] = *reinterpret_cast<const uint2*>(kp + 8 * s);
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const int d = (tid + e * kWaves * 64) >> 2;
      if (D % 64 == 0 || d < D) vc[e] = ldg16(vp + int64_t(d) * P);
    }
    ks = c.k_scales[int64_t(spage) * c.H + head];
    vs = c.v_scales[int64_t(spage) * c.H + head];
  };
  const auto store = [&](uint8_t* to) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      *reinterpret_cast<bf16x8*>(to + key_row * kKeyRow + piece * (D / 2) + 16 * s) = codes_bf16<FMT>(kc[s].x, kc[s].y);
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const int d = (tid + e * kWaves * 64) >> 2;
      if (D % 64 != 0 && d >= D) break;
      const u32x4 v = live >= 16 ? vc[e] : live_codes(vc[e], live);
      f16x8* at = reinterpret_cast<f16x8*>(to + kKeys + d * kValueRow + piece * 32);
      at[0] = codes_f16<FMT>(v[0], v[1]);
      at[1] = codes_f16<FMT>(v[2], v[3]);
    }
  };
  int blk = sh.first + part * sh.each;
  if (blk < end) load(blk);

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
    uint8_t* at = lds[buffer];
    store(at);
    float f = ks * c.scale_log2;
    const float lv = there ? log2f(vs) : -INFINITY;
    const bool here = there;
    if (blk + 1 < end) load(blk + 1);
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
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(at + (16 * i + col) * kKeyRow + quarter * (D / 2) + 16 * s);
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
        const f16x8 vf = *reinterpret_cast<const f16x8*>(at + kKeys + (16 * t + col) * kValueRow + quarter * 32 + 16 * u);
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
