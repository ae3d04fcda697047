// attention_tile.hip -- attention over the paged 8-bit cache for many rows: prompts, pieces of prompts, many query heads to a
// head of the cache.
//
// What bounds it is arithmetic: two products of 2 D operations each a (row, position), 2^x, sums and conversions beside them. A
// workgroup takes 128 rows of one head of the cache of one sequence, 32 for each of its four waves, and all waves walk
// the same blocks of 64 positions. A block's codes are asked for from memory while the block before is worked on, converted
// once by the whole workgroup (keys to bf16, values to fp16), and handed to the waves through two LDS buffers in turn, so
// that there is one barrier a block. Products, lane layout and softmax are those of the few-row kernel. Measured, with the kernel of
// 256 rows below where it serves: 4 prompts of 4500, 32 heads on 8 of 128, e4m3: 468 us, 940 TFLOP/s; 1024 tokens, 64 heads
// on 8, INT8, on 30000 positions: 874 us, 1.17 PFLOP/s (a bf16 matrix product of 8192 reaches 1.44, of 16384 1.62). 4 prompts of up to 4500 and
// that piece with this kernel's other head sizes, in TFLOP/s: 64: 690 and 670, 96: 730 and 820, 192: 500 and 590, 256: 490 and 580 (192 and 256
// leave room for one workgroup a CU, one wave a SIMD, so that nothing hides softmax and barriers).
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
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  __builtin_amdgcn_sched_barrier(0);
}

// A workgroup's part of the work. One sequence after the other, its last tiles first, which see most. Heads next to each other: with
// eight of them a head's workgroups run on one XCD, whose L2 then holds one head of one or two sequences (with all sequences' tiles
// in turn instead, 4 prompts of 4500 took 690 us at a build where they take 505 so).
struct Place {
  int head, b, part, r0;
};

__device__ __forceinline__ Place place_of(const KvCall& c, int tile_rows) {
  const unsigned heads = unsigned(c.H), parts = unsigned(c.n_split);
  const unsigned tile = (gridDim.x - 1 - blockIdx.x) / (heads * parts);
  return {int(blockIdx.x % heads), int(blockIdx.y), int(blockIdx.x / heads % parts), int(tile) * tile_rows};
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

// The order of a product's instructions: six LDS reads first, then two matrix instructions for each further read, so that a read's
// result is waited for while others are on their way.
template <int READS>
__device__ __forceinline__ void reads_ahead() {
  constexpr int kAhead = 6;
  __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
  for (int g = 0; g < READS - kAhead; ++g) {
    __builtin_amdgcn_sched_group_barrier(0x008, kNQ, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, kNQ * kAhead, 0);
}

// A wave's rows, r = w0 .., to out, or to the parts.
template <int D>
__device__ __forceinline__ void write_rows(const KvCall& c, const KvSeq& sq, const Share& sh, int b, int head, int part, int w0, int rows,
                                           const Rows<kNQ, D / 16>& st) {
  const int lane = threadIdx.x & 63, col = lane & 15, quarter = lane >> 4;
#pragma unroll
  for (int n = 0; n < kNQ; ++n) {
    const int r = w0 + 16 * n + col;
    const float total = row_sum(st.sum[n]), by = lowered(total), to = unit(st.rel[n]) * (sh.parts == 1 ? 1.0f : kKept);
    if (r >= rows) continue;
    const int i = r / c.G, h = head * c.G + r % c.G;
    if (sh.parts == 1) {
      auto* out = static_cast<uint16_t*>(c.out) + ((int64_t(sq.first) + i) * c.Hq + h) * D + 4 * quarter;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        const f32x4& o = st.acc[n][t];
        *reinterpret_cast<uint2*>(out + 16 * t) =
            make_uint2(f32x2_to_bf16x2_rne(o[0] * by * to, o[1] * by * to), f32x2_to_bf16x2_rne(o[2] * by * to, o[3] * by * to));
      }
    } else {
      const int64_t at = part_row(c, sq, b, i, h) + part;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        f32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = st.acc[n][t][j] * by * to;
        *reinterpret_cast<f32x4*>(c.ws_o + at * D + 16 * t + 4 * quarter) = o;
      }
      if (quarter == 0) *reinterpret_cast<float2*>(c.ws_ml + 2 * at) = make_float2(st.top[n], total);
    }
  }
}

template <int D, int FMT>
__global__ __launch_bounds__(kWaves * 64, D <= 128 ? 2 : 1) void attention_tile_kernel(KvCall c) {
  constexpr int kSteps = D / 32, kTiles = D / 16;
  constexpr int kKeys = (D & (D - 1)) == 0 ? kBlock * D * 2 : 4 * kBlock * (D / 32 | 1) * 16;
  constexpr int kBuffer = kKeys + D * kBlock * 2;
  constexpr int kPieces = (D * 4 + kWaves * 64 - 1) / (kWaves * 64);    // 16-byte pieces of values a thread stages
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kBuffer];
  const Place place = place_of(c, kTileRows);
  const int head = place.head, b = place.b, part = place.part, r0 = place.r0;
  const KvSeq sq = attention_sequence(c, b);
  const int rows = sq.n * c.G;
  if (r0 >= rows) return;
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
  int kpage = 0, vpage = 0, spage = 0;     // of the wave's keys, the thread's values, the lane's positions in the blocks loaded next
  uint2 kc[kSteps];
  u32x4 vc[kPieces];
  int live;                // positions of this thread's values that exist
  float ks, vs;            // scales of this lane's positions
  bool there;
  int zero;     // (vector loads of the pages: a scalar one would be waited for at the next barrier, with the LDS writes)
  asm volatile("v_mov_b32 %0, 0" : "=v"(zero));
  const auto page_of = [&](int position) { return table[(min(position, sq.len - 1) + zero) >> shift]; };     // (past the end: the last page, not used)
  const uint32_t key_offset = unsigned(((head << shift) + (key & 15)) * D + piece * (D / 4));
  const uint8_t* const vp = static_cast<const uint8_t*>(c.v_pages) + ((int64_t(head) * D + (tid >> 2)) << shift);
  const auto load_codes = [&](int blk) {
    const int vg = blk * kBlock + 16 * piece;
    live = unsigned(vpage) < unsigned(c.num_pages) ? sq.len - vg : 0;
    const uint32_t from = live > 0 ? vpage : 0, wanted = __builtin_amdgcn_readfirstlane(kpage), page = wanted < unsigned(c.num_pages) ? wanted : 0;
    const uint8_t* k = static_cast<const uint8_t*>(c.k_pages) + uint64_t(page) * c.page_bytes + ((blk * kBlock + 16 * wave) & (P - 1)) * D;
    const uint8_t* v = vp + uint64_t(from) * c.page_bytes + (vg & (P - 1));
#pragma unroll
    for (int s = 0; s < kSteps; ++s) kc[s] = *reinterpret_cast<const uint2*>(k + key_offset + 8 * s);
#pragma unroll
    for (int e = 0; e < kPieces; ++e)
      if (D % 64 == 0 || (tid >> 2) + 64 * e < D) vc[e] = ldg16(v + (int64_t(64 * e) << shift));
  };
  const auto load_scales = [&](int blk) {
    there = blk * kBlock + 16 * quarter < sq.len && unsigned(spage) < unsigned(c.num_pages);
    const uint64_t at = uint64_t(there ? spage : 0) * unsigned(c.H) + unsigned(head);
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
  const auto load_code_pages = [&](int at) {
    kpage = page_of(at * kBlock + 16 * wave);
    vpage = page_of(at * kBlock + 16 * piece);
  };
  const int w0 = r0 + wave * 16 * kNQ;      // the wave's first row
  bf16x8 qf[kNQ][kSteps];
  load_queries(c, sq, head, w0, rows, qf);
  if (blk < end) {
    load_code_pages(blk);
    spage = page_of(blk * kBlock + 16 * quarter);
    load_codes(blk);
    load_scales(blk);
    load_code_pages(blk + 1);
    spage = page_of((blk + 1) * kBlock + 16 * quarter);
  }

  int pos[kNQ];
#pragma unroll
  for (int n = 0; n < kNQ; ++n) {
    const int r = w0 + 16 * n + col;
    pos[n] = r < rows ? before + r / c.G : -1;
  }
  const int pos_first = before + w0 / c.G;
  const int pos_last = w0 < rows ? before + (min(w0 + 16 * kNQ, rows) - 1) / c.G : -1;

  sign_queries(c, qf);

  Rows<kNQ, kTiles> st;
  st.clear();
  for (int buffer = 0; blk < end; ++blk, buffer ^= 1) {
    uint8_t* at = lds + buffer * kBuffer;
    store(at);
    load_codes(blk + 1);
    load_code_pages(blk + 2);
    lds_barrier();
    const int base = blk * kBlock, vg = base + 16 * quarter;
    // (blocks that none of the wave's rows sees are left out)
    if (base <= pos_last && (c.window == 0 || base + kBlock - 1 > pos_first - c.window)) {
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
      reads_ahead<4 * kSteps>();
      float f = ks * c.scale_log2;
      const float lv = there ? log2f(vs) : -INFINITY;
      if (base + kBlock - 1 > pos_first || (c.window > 0 && base <= pos_last - c.window) || __any(!there)) {
        mask_scores<kNQ>(score, pos, vg, c.window, there, f);
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
      reads_ahead<2 * kTiles>();
    }
    // (after the last use of this block's: into the same registers, without a copy that would wait for them)
    load_scales(blk + 1);
    spage = page_of((blk + 2) * kBlock + 16 * quarter);
  }

  write_rows<D>(c, sq, sh, b, head, part, w0, rows, st);
}

// Eight waves, 32 rows each, two on a SIMD: waves 0-3 and 4-7 half a turn apart, so that one wave of a SIMD multiplies (values of block
// k - 1, keys of block k) while the other has its maxima and exponentials. A barrier ends each half. Between its matrix instructions
// every wave converts its share of the keys of k + 1 and the values of k, and asks for the next: a half turn before their first
// reader's turn, into the one of two LDS buffers that its last reader left a half turn before.
// The multiplying wave goes first where both could issue (1024 x 8 rows on 30000 at one build: 897 us, 970 without). What bounds it is the
// vector instructions' port: 150 a wave and block for the softmax, 90 for conversions and addresses, beside 64 matrix instructions;
// without its products that build took 653 us, without softmax 777, without staging 720, products and LDS reads alone 618.
// Head size 128 alone: larger ones leave no room for two waves on a SIMD, at 64 three workgroups of the kernel above do better
// (2048 rows of 8 heads on 30000: 1443 us, 1632 here).
template <int FMT>
__global__ __launch_bounds__(512, 2) void attention_paired_kernel(KvCall c) {
  constexpr int D = 128;
  constexpr int kSteps = D / 32, kTiles = D / 16, kRows = 8 * 16 * kNQ;
  constexpr int kKeys = kBlock * D * 2, kValues = D * kBlock * 2;
  constexpr int kProducts = 2 * kTiles + 4 * kSteps;
  constexpr int kChunks = 2;                                            // 16-byte chunks of bf16 keys a thread stages
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * (kKeys + kValues)];
  const Place place = place_of(c, kRows);
  const int head = place.head, b = place.b, part = place.part, r0 = place.r0;
  const KvSeq sq = attention_sequence(c, b);
  const int rows = sq.n * c.G;
  if (r0 >= rows) return;
  const Share sh = share_of(c, sq, r0, kRows);
  if (part >= sh.parts) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, col = lane & 15, quarter = lane >> 4;
  const int shift = c.page_shift, P = 1 << shift;
  const int before = sq.len - sq.n, most = sq.len - 1;
  const int first = sh.first + part * sh.each, end = min(first + sh.each, sh.end);
  const int32_t* table = c.table + int64_t(b) * c.width;

  // Staging: a thread takes an eighth of one key's channels (the 8 keys of a wave are of one page, whose address is scalar), and one
  // 16-byte piece of values (channel, 16 positions).
  const int key = tid >> 3, eighth = tid & 7, piece = tid & 3;
  const int key_row = 16 * ((key >> 2) & 3) + 4 * (key >> 4) + (key & 3);
  uint2 kc[kChunks];
  u32x4 vc;
  int live = 16;                        // positions of this thread's values that exist
  float ks = 0, vs = 0;                 // scales of this lane's positions
  bool there = false;
  int kpage = 0, vpage = 0, spage = 0;
  // Page of a position (past the end: the last page, not used). Asked for by vector loads, the wave's own too: a scalar one would be
  // waited for at the next barrier, with the LDS writes.
  int zero;
  asm volatile("v_mov_b32 %0, 0" : "=v"(zero));
  const auto page_of = [&](int position) {
    return *reinterpret_cast<const int32_t*>(reinterpret_cast<const uint8_t*>(table) + ((unsigned(min(position, most) + zero) >> shift) << 2));
  };
  uint32_t key_offset = unsigned(((head << shift) + (key & 15)) * D + eighth * (D / 8));
  const uint8_t* const vp = static_cast<const uint8_t*>(c.v_pages) + ((int64_t(head) * D + (tid >> 2)) << shift);
  const auto load_keys = [&](int blk) {
    const uint32_t from = __builtin_amdgcn_readfirstlane(kpage);
    const uint32_t page = from < unsigned(c.num_pages) ? from : 0;
    const uint8_t* k = static_cast<const uint8_t*>(c.k_pages) + uint64_t(page) * c.page_bytes + ((blk * kBlock + 16 * (wave >> 1)) & (P - 1)) * D;
#pragma unroll
    for (int s = 0; s < kChunks; ++s) kc[s] = *reinterpret_cast<const uint2*>(k + key_offset + 8 * s);
  };
  const auto load_values = [&](int blk) {
    const int vg = blk * kBlock + 16 * piece;
    live = unsigned(vpage) < unsigned(c.num_pages) ? sq.len - vg : 0;
    const uint32_t from = live > 0 ? vpage : 0;
    vc = ldg16(vp + uint64_t(from) * c.page_bytes + (vg & (P - 1)));
  };
  const auto load_scales = [&](int blk) {
    there = blk * kBlock + 16 * quarter <= most && unsigned(spage) < unsigned(c.num_pages);
    const uint32_t at = (unsigned(there ? spage : 0) * unsigned(c.H) + unsigned(head)) << 2;     // (below 2^32: a page's codes are at least 1024 a head)
    ks = *reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(c.k_scales) + at);
    vs = *reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(c.v_scales) + at);
  };
  // Places in LDS, of the buffers in turn: two of keys, then two of values. Chunk s of a key row, half u of a channel is at ^ 16 s.
  uint32_t k_read = key_at<D>(col, quarter, 0), k_write = key_at<D>(key_row, eighth / 2, eighth % 2 * kChunks);
  uint32_t v_read = 2 * kKeys + value_at(col, quarter, 0), v_write = 2 * kKeys + value_at(tid >> 2, piece, 0);
  // (opaque where they are converted: the conversions stay among the matrix instructions they stand between)
  const auto store_keys = [&](int s) {
    asm volatile("" : "+v"(kc[s].x), "+v"(kc[s].y));
    *reinterpret_cast<bf16x8*>(lds + (k_write ^ (16u * s))) = codes_bf16<FMT>(kc[s].x, kc[s].y);
  };
  const auto store_values = [&](int u) {
    uint32_t lo = vc[2 * u], hi = vc[2 * u + 1];
    asm volatile("" : "+v"(lo), "+v"(hi));
    *reinterpret_cast<f16x8*>(lds + (v_write ^ (16u * u))) = codes_f16<FMT>(lo, hi);
  };

  const int w0 = r0 + wave * 16 * kNQ;      // the wave's first row
  bf16x8 qf[kNQ][kSteps];
  load_queries(c, sq, head, w0, rows, qf);
  int pos[kNQ];
#pragma unroll
  for (int n = 0; n < kNQ; ++n) {
    const int r = w0 + 16 * n + col;
    pos[n] = r < rows ? before + r / c.G : -1;
  }
  const int pos_first = before + w0 / c.G;
  const int pos_last = w0 < rows ? before + (min(w0 + 16 * kNQ, rows) - 1) / c.G : -1;

  Rows<kNQ, kTiles> st;
  st.clear();
  if (first < end) {
    kpage = page_of(first * kBlock + 16 * (wave >> 1));
    vpage = page_of(first * kBlock + 16 * piece);
    spage = page_of(first * kBlock + 16 * quarter);
    load_keys(first);
    load_values(first);
    kpage = page_of((first + 1) * kBlock + 16 * (wave >> 1));
    vpage = page_of((first + 1) * kBlock + 16 * piece);
    store_keys(0);
    store_keys(1);
    k_write ^= kKeys;
    v_read ^= kValues;
    load_keys(first + 1);
    kpage = page_of((first + 2) * kBlock + 16 * (wave >> 1));
    f32x4 score[kNQ][4];
    f16x8 weight[kNQ][2] = {};          // of block k - 1; none before the first, whose place in LDS holds zeros
    *reinterpret_cast<u32x4*>(lds + (v_write ^ kValues)) = u32x4{0, 0, 0, 0};
    *reinterpret_cast<u32x4*>(lds + (v_write ^ kValues ^ 16u)) = u32x4{0, 0, 0, 0};
    sign_queries(c, qf);
    lds_barrier();
    if (wave >= 4) lds_barrier();
    for (int blk = first; blk <= end; ++blk) {
      // The turn's products in 32 steps, a 16-byte piece of LDS and two matrix instructions each: values of k - 1, then keys of k.
      const auto read = [&](int j) {
        return *reinterpret_cast<const u32x4*>(j < kProducts / 2 ? lds + (v_read ^ (16u * (j / kTiles))) + 16 * (j % kTiles) * 128
                                                                 : lds + (k_read ^ (16u * ((j - kProducts / 2) / 4))) + 16 * (j % 4) * D * 2);
      };
      const auto multiply = [&](int j, u32x4 x) {
#pragma unroll
        for (int n = 0; n < kNQ; ++n) {
          if (j < kProducts / 2) {
            st.acc[n][j % kTiles] = mfma_f16(__builtin_bit_cast(f16x8, x), weight[n][j / kTiles], st.acc[n][j % kTiles]);
          } else {
            const int i = j % 4, s = (j - kProducts / 2) / 4;
            score[n][i] = mfma_bf16(__builtin_bit_cast(bf16x8, x), qf[n][s], s ? score[n][i] : f32x4{0, 0, 0, 0});
          }
        }
      };
      // The wave's share of the staging, in pieces to go between (past the range's end too, where nothing reads what is stored).
      const auto stage = [&](int piece_of_work) {
        switch (piece_of_work) {
          case 0:
            load_scales(blk);
            spage = page_of((blk + 1) * kBlock + 16 * quarter);
            break;
          case 1: store_keys(0); break;
          case 2: store_keys(1); break;
          case 3:
            load_keys(blk + 2);
            kpage = page_of((blk + 3) * kBlock + 16 * (wave >> 1));
            break;
          case 4: store_values(0); break;
          case 5: store_values(1); break;
          case 6:
            load_values(blk + 1);
            vpage = page_of((blk + 2) * kBlock + 16 * piece);
            break;
        }
      };
      asm volatile("" : "+v"(key_offset));      // (an offset to a scalar address, not widened ahead of the loop)
      if (__any(live < 16)) vc = live_codes(vc, live);
      __builtin_amdgcn_s_setprio(1);
      // four steps at a time, the next four's pieces asked for before, the staging's vector instructions between
      u32x4 x[4], y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = read(j);
#pragma unroll
      for (int r = 0; r < kProducts / 4; ++r) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r + 1 < kProducts / 4) y[j] = read(4 * r + 4 + j);
        stage(r);
#pragma unroll
        for (int j = 0; j < 4; ++j) multiply(4 * r + j, x[j]);
        if (r + 1 < kProducts / 4) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
        for (int j = 0; j < 4 * kNQ; ++j) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = y[j];
      }
      __builtin_amdgcn_s_setprio(0);
      lds_barrier();
      if (blk < end) {
        const int base = blk * kBlock;
        float f = ks * c.scale_log2;
        const float lv = there ? log2f(vs) : -INFINITY;
        if (base + kBlock - 1 > pos_first || (c.window > 0 && base <= pos_last - c.window) || __any(!there)) {
          mask_scores<kNQ>(score, pos, base + 16 * quarter, c.window, there, f);
          f = 1.0f;
        }
        st.step(score, f, lv, weight);
      }
      lds_barrier();
      k_read ^= kKeys;
      k_write ^= kKeys;
      v_read ^= kValues;
      v_write ^= kValues;
    }
    if (wave < 4) lds_barrier();
  }

  write_rows<D>(c, sq, sh, b, head, part, w0, rows, st);
}

template <int D, int FMT>
hipError_t go(const KvCall& c, hipStream_t s) {
  const int64_t rows = int64_t(c.hi_n) * c.G;
  const int64_t tiles = (rows + c.tile_rows - 1) / c.tile_rows;
  const dim3 grid(unsigned(c.H) * unsigned(c.n_split) * unsigned(tiles), unsigned(c.B));
  if constexpr (D == 128) {
    if (c.tile_rows == 2 * kTileRows) {
      hipLaunchKernelGGL((attention_paired_kernel<FMT>), grid, dim3(512), 0, s, c);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((attention_tile_kernel<D, FMT>), grid, dim3(kWaves * 64), 0, s, c);
  return hipGetLastError();
}

template <int D>
hipError_t pick(const KvCall& c, hipStream_t s) {
  return c.fmt == HQ_KV_INT8 ? go<D, HQ_KV_INT8>(c, s) : go<D, HQ_KV_FP8_E4M3>(c, s);
}

}  // namespace

hipError_t launch_attention_tiles(const KvCall& c, hipStream_t s) {
  switch (c.D) {
    case 64: return pick<64>(c, s);
    case 96: return pick<96>(c, s);
    case 128: return pick<128>(c, s);
    case 192: return pick<192>(c, s);
    default: return pick<256>(c, s);
  }
}

}  // namespace hq
