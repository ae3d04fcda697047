// attention.hip -- attention over the paged 8-bit cache for few rows: softmax(sm_scale * q . k) v with the running maximum
// and sum of each row, one pass over the keys and values, read once for all the query heads and tokens that share them.
//
// What bounds it is the reading of the cache. A workgroup takes up to 32 rows (one head of the cache of one sequence) and a
// range of the positions; its four waves take blocks of 64 positions in turn and join their results through LDS. The
// positions are split over workgroups as well, and a second launch joins the parts.
//
// Codes go from memory to the matrix instructions without a pass through LDS:
//   S^T = K . Q^T    tile i of 4: A row m is position 16 (m / 4) + 4 i + (m % 4) of the block; a lane loads a quarter of a
//                    key's channels (their order inside a dot product is free);
//   O^T += V^T . P^T A row m is channel 16 t + m, whose 16 codes of the lane's positions are one 16-byte load from the
//                    transposed page; P^T is what the lane already holds.
// The next block's keys are asked for when this one's are used up, and so the values: the loads of one block are in flight
// while the other is worked on, in the same registers (a whole block ahead in registers of its own was no faster).
//
// Measured (a 2 GiB copy moves 5.05 TB/s, a read stream 6.13; kernels alone, in a trace): one token, 32 heads on 8, 131071
// positions: 269 MB in 50 us, 5.4 TB/s, and 5 us for the join; 64 tokens on lengths up to 8000 (INT8, 64 heads on 8): 141 us, 4.8
// TB/s, the rest is the longest sequences' tail. One token on 100 positions: 5.3 us, a launch and three dependent trips to memory.
// 32 rows at head sizes 192 and 256 spill up to 4 registers.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention_ops.h"

namespace hq {

namespace {

constexpr int kWaves = 4;
constexpr int kFewRows = 32;     // rows of a head that one workgroup takes here; more go to the tiled kernel
constexpr int kTileRows = 128;   // rows of a workgroup of the tiled kernel, of its paired form twice that
constexpr int kMaxSplit = 128;

template <int D, int FMT, int NQ>
__global__ __launch_bounds__(kWaves * 64, D <= 128 ? 2 : 1) void attention_kernel(KvCall c) {
  constexpr int kSteps = D / 32;      // matrix instructions of a dot product
  constexpr int kTiles = D / 16;      // 16-channel tiles of the output
  const int b = blockIdx.y;
  const KvSeq sq = attention_sequence(c, b);
  // heads next to each other, so that with eight of them a head's workgroups run on one XCD and share its L2
  const int head = int(blockIdx.x % unsigned(c.H)), part = int(blockIdx.x / unsigned(c.H) % unsigned(c.n_split));
  const int r0 = int(blockIdx.x / unsigned(c.H) / unsigned(c.n_split)) * 16 * NQ;
  const int rows = sq.n * c.G;
  if (r0 >= rows) return;
  const Share sh = share_of(c, sq, r0, 16 * NQ);
  if (part >= sh.parts) return;
  // the wave is the same for all its lanes: blocks, addresses and branches that go by it are scalar
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, quarter = lane >> 4;
  const int shift = c.page_shift, P = 1 << shift;
  const int before = sq.len - sq.n;

  // codes and scales of one of the wave's blocks, and the pages of the block that is asked for next
  struct Codes {
    uint2 k[4][kSteps];
    u32x4 v[kTiles];
    float ks, vs;
    bool there;      // the page of the 16 positions whose values the lane holds
  };
  const auto* kp = static_cast<const uint8_t*>(c.k_pages);
  const auto* vp = static_cast<const uint8_t*>(c.v_pages);
  const int32_t* table = c.table + int64_t(b) * c.width;
  const int end = min(sh.first + (part + 1) * sh.each, sh.end);
  int blk = sh.first + part * sh.each + wave;
  int kpage, vpage;      // of the 16 positions whose keys this lane loads, and of those whose values it holds
  const auto load_pages = [&](int at) {
    const int kg = at * kBlock + 16 * (col >> 2), vg = at * kBlock + 16 * quarter;
    kpage = at < end && kg < sq.len ? table[kg >> shift] : -1;
    vpage = at < end && vg < sq.len ? table[vg >> shift] : -1;
  };
  const auto load_keys = [&](int at, Codes& to) {
    const int kg = at * kBlock + 16 * (col >> 2);
    const uint32_t page = unsigned(kpage) < unsigned(c.num_pages) ? kpage : 0;
    const uint8_t* p = kp + uint64_t(page) * c.page_bytes + ((head << shift) + (kg & (P - 1)) + (col & 3)) * D + quarter * (D / 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) to.k[i][s] = *reinterpret_cast<const uint2*>(p + 4 * i * D + 8 * s);
  };
  const auto load_values = [&](int at, Codes& to) {
    const int vg = at * kBlock + 16 * quarter;
    to.there = unsigned(vpage) < unsigned(c.num_pages);
    // (a page that does not exist stands for page 0, whose scales may be anything)
    const uint32_t page = to.there ? vpage : 0;
    const uint8_t* p = vp + uint64_t(page) * c.page_bytes + (((head * D + col) << shift) + (vg & (P - 1)));
#pragma unroll
    for (int t = 0; t < kTiles; ++t) to.v[t] = ldg16(p + ((16 * t) << shift));
    const uint64_t scale = uint64_t(page) * unsigned(c.H) + unsigned(head);
    to.ks = c.k_scales[scale];
    to.vs = c.v_scales[scale];
  };
  load_pages(blk);

  // this lane's rows, one of each 16: query fragments and the last position seen
  bf16x8 qf[NQ][kSteps];
  load_queries(c, sq, head, r0, rows, qf);
  int pos[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = r0 + 16 * n + col;
    pos[n] = r < rows ? before + r / c.G : -1;
  }
  const int pos_first = before + r0 / c.G, pos_last = before + (min(r0 + 16 * NQ, rows) - 1) / c.G;

  Rows<NQ, kTiles> st;
  st.clear();
  // A block's turn. `keys_done` runs when its keys are used up.
  const auto turn = [&](int at, Codes& x, auto keys_done) {
    const int base = at * kBlock, vg = base + 16 * quarter;
    f32x4 score[NQ][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) score[n][i] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const bf16x8 kf = codes_bf16<FMT>(x.k[i][s].x, x.k[i][s].y);
#pragma unroll
        for (int n = 0; n < NQ; ++n) score[n][i] = mfma_bf16(kf, qf[n][s], score[n][i]);
      }
    }
    keys_done();
    float f = x.ks * c.scale_log2;
    const float lv = x.there ? log2f(x.vs) : -INFINITY;
    if (base + kBlock - 1 > pos_first || (c.window > 0 && base <= pos_last - c.window) || __any(!x.there)) {
      mask_scores<NQ>(score, pos, vg, c.window, x.there, f);
      f = 1.0f;
      const int live = x.there ? sq.len - vg : 0;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) x.v[t] = live_codes(x.v[t], live);
    }
    f16x8 weight[NQ][2];
    st.step(score, f, lv, weight);
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f16x8 vf = codes_f16<FMT>(x.v[t][2 * u], x.v[t][2 * u + 1]);
#pragma unroll
        for (int n = 0; n < NQ; ++n) st.acc[n][t] = mfma_f16(vf, weight[n][u], st.acc[n][t]);
      }
  };
  Codes x;
  if (blk < end) {
    load_keys(blk, x);
    load_values(blk, x);
    load_pages(blk + kWaves);
  }
  sign_queries(c, qf);
  // the next block's keys into the registers of this one's as soon as they are used up, and so its values
  for (; blk < end; blk += kWaves) {
    turn(blk, x, [&] {
      if (blk + kWaves < end) load_keys(blk + kWaves, x);
    });
    if (blk + kWaves < end) {
      load_values(blk + kWaves, x);
      load_pages(blk + 2 * kWaves);
    }
  }

  // the four waves' parts, joined 16 rows at a time: sums to the largest of their references, and the average from there
  __shared__ float tops[kWaves][16], rels[kWaves][16], sums[kWaves][16];
  __shared__ float parts[kWaves][16][D + 4];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const float l = row_sum(st.sum[n]);
    if (n) __syncthreads();
    if (quarter == 0) {
      tops[wave][col] = st.top[n];
      rels[wave][col] = st.rel[n];
      sums[wave][col] = l;
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) *reinterpret_cast<f32x4*>(&parts[wave][col][16 * t + 4 * quarter]) = st.acc[n][t];
    __syncthreads();
    // a lane's own row and wave: its factor, and what makes the row's sum an average
    const float top = row_max(tops[quarter][col]), below = tops[quarter][col] - top, at = below + rels[quarter][col], ref = row_max(at);
    const float factor = exp2_fast(at - ref), total = row_sum(exp2_fast(below) * sums[quarter][col]);
    const float by = lowered(total), to = unit(ref) * (sh.parts == 1 ? 1.0f : kKept);
    for (int e = threadIdx.x; e < 16 * (D / 4); e += kWaves * 64) {
      const int row = e / (D / 4), d = (e % (D / 4)) * 4;
      const int r = r0 + 16 * n + row;
      f32x4 o = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __shfl(factor, row + 16 * w, 64);
        const f32x4 x = *reinterpret_cast<const f32x4*>(&parts[w][row][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += f * x[j];
      }
      const float row_by = __shfl(by, row, 64), row_to = __shfl(to, row, 64);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = o[j] * row_by * row_to;
      const float2 ml = make_float2(__shfl(top, row, 64), __shfl(total, row, 64));
      if (r >= rows) continue;
      const int i = r / c.G, h = head * c.G + r % c.G;
      if (sh.parts == 1) {
        const uint2 w = {f32x2_to_bf16x2_rne(o[0], o[1]), f32x2_to_bf16x2_rne(o[2], o[3])};
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.out) + ((int64_t(sq.first) + i) * c.Hq + h) * D + d) = w;
      } else {
        const int64_t slot = part_row(c, sq, b, i, h) + part;
        *reinterpret_cast<f32x4*>(c.ws_o + slot * D + d) = o;
        if (d == 0) *reinterpret_cast<float2*>(c.ws_ml + 2 * slot) = ml;
      }
    }
  }
}

// The parts of a row joined: one workgroup a (token, query head), its waves taking parts in turn, a lane D / 64 channels.
template <int D>
__global__ __launch_bounds__(kWaves * 64) void attention_join_kernel(KvCall c, int tile_rows) {
  constexpr int kEach = (D + 63) / 64;
  __shared__ float parts[kWaves][kEach * 64];
  const int b = blockIdx.y;
  const KvSeq sq = attention_sequence(c, b);
  const int head = int(blockIdx.x % unsigned(c.H)), r = int(blockIdx.x / unsigned(c.H));
  if (r >= sq.n * c.G) return;
  const Share sh = share_of(c, sq, r / tile_rows * tile_rows, tile_rows);
  if (sh.parts == 1) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int i = r / c.G, h = head * c.G + r % c.G;
  const int64_t at = part_row(c, sq, b, i, h);
  static_assert(kMaxSplit <= 2 * 64, "a lane holds two parts' maxima");
  const float2 none = make_float2(-INFINITY, 0.0f);
  const auto* all = reinterpret_cast<const float2*>(c.ws_ml) + at;
  const float2 ml0 = lane < sh.parts ? all[lane] : none, ml1 = lane + 64 < sh.parts ? all[lane + 64] : none;
  constexpr int kAhead = 4;   // parts asked for together, the first of them before the shares are known
  float x[kAhead][kEach];
  const auto load = [&](int s0) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int s = s0 + a * kWaves;
        x[a][j] = s < sh.parts && (D % 64 == 0 || lane + 64 * j < D) ? c.ws_o[(at + s) * D + lane + 64 * j] : 0.0f;
      }
  };
  load(wave);
  float m = fmaxf(ml0.x, ml1.x);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  float f0 = exp2_fast(ml0.x - m) * ml0.y, f1 = exp2_fast(ml1.x - m) * ml1.y, total = f0 + f1;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) total += __shfl_xor(total, off, 64);
  const float whole = inverse(total) * (1.0f / kKept);
  f0 *= whole;
  f1 *= whole;
  float o[kEach] = {};
  for (int s0 = wave; s0 < sh.parts; s0 += kAhead * kWaves) {
    if (s0 != wave) load(s0);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int s = s0 + a * kWaves;
      if (s >= sh.parts) break;
      const float f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s < 64 ? f0 : f1), s & 63));
#pragma unroll
      for (int j = 0; j < kEach; ++j) o[j] += f * x[a][j];
    }
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) parts[wave][lane + 64 * j] = o[j];
  __syncthreads();
  auto* out = static_cast<uint16_t*>(c.out) + ((int64_t(sq.first) + i) * c.Hq + h) * D;
  for (int d = threadIdx.x; d < D; d += kWaves * 64) out[d] = f32_to_bf16_rne((parts[0][d] + parts[1][d]) + (parts[2][d] + parts[3][d]));
}

template <int D>
hipError_t join(const KvCall& c, int tile_rows, hipStream_t s) {
  const int64_t rows = int64_t(c.hi_n) * c.G;
  if (c.n_split > 1)
    hipLaunchKernelGGL((attention_join_kernel<D>), dim3(unsigned(rows) * unsigned(c.H), unsigned(c.B)), dim3(kWaves * 64), 0, s, c, tile_rows);
  return hipGetLastError();
}

template <int D, int FMT>
hipError_t go(const KvCall& c, bool wide, hipStream_t s) {
  const int rows = wide ? 32 : 16;
  const dim3 grid(unsigned((c.hi_n * c.G + rows - 1) / rows) * unsigned(c.n_split) * unsigned(c.H), unsigned(c.B));
  if (wide) hipLaunchKernelGGL((attention_kernel<D, FMT, 2>), grid, dim3(kWaves * 64), 0, s, c);
  else hipLaunchKernelGGL((attention_kernel<D, FMT, 1>), grid, dim3(kWaves * 64), 0, s, c);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? join<D>(c, rows, s) : e;
}

template <int D>
hipError_t pick(const KvCall& c, bool wide, hipStream_t s) {
  return c.fmt == HQ_KV_INT8 ? go<D, HQ_KV_INT8>(c, wide, s) : go<D, HQ_KV_FP8_E4M3>(c, wide, s);
}

}  // namespace

int64_t attention_groups(const KvCall& c) { return (int64_t(c.max_new) * c.G + kTileRows - 1) / kTileRows * c.H * c.B; }

namespace {
// Parts of the positions: no more workgroups than run at once, each with at least `least` blocks. With more, the last ones
// run alone: one token on 131071 positions with 256 / 512 / 768 / 1024 workgroups 57.9 / 57.5 / 59.3 / 60.1 us; 16 tokens on up to
// 30000 140.5 / 139.6 / 158.6 / 142.2 (134.3 with 2048); D = 64, 16 on up to 10000 38.0 / 31.4 / 32.6 / 32.4; D = 192, 32 on up to 4000 65.2 /
// 66.4 / 70.8 / 69.1; D = 256, 4 tokens on 20000 with 256 / 512 / 1024: 23.8 / 32.1 / 38.4.
void split_of(int64_t groups, int64_t wanted, int64_t least, int64_t max_kv, int* n_split, int* each) {
  const int64_t blocks = std::max<int64_t>((max_kv + kBlock - 1) / kBlock, 1);
  int64_t n = std::max<int64_t>(wanted / groups, 1);
  n = std::min<int64_t>(std::min(n, (blocks + least - 1) / least), kMaxSplit);
  *each = int((blocks + n - 1) / n);
  *n_split = int(n);
}
}  // namespace

AttentionPlan plan_attention(const KvCall& c, int64_t max_kv) {
  AttentionPlan p{};
  const int64_t most = int64_t(c.max_new) * c.G;
  // what a workgroup's rows see, at most; a window may begin and end inside a block
  if (c.window > 0) max_kv = std::min(max_kv, int64_t(c.window) + std::min<int64_t>(c.max_new, 256) + kBlock);
  // sequences with few rows among others with many have their own launch
  p.few = most <= kFewRows ? c.max_new : c.B > 1 ? kFewRows / c.G : 0;
  p.many = c.max_new > p.few;
  size_t at = 0;
  const auto room = [&](int64_t slots, int n_split, size_t* o, size_t* ml) {
    if (n_split == 1) return;
    *o = at;
    *ml = at + size_t(slots) * c.Hq * n_split * c.D * 4;
    at = *ml + (size_t(slots) * c.Hq * n_split * 8 + 15) / 16 * 16;
  };
  if (p.few) {
    const int resident = c.D > 192 ? 256 : 512;      // two workgroups a CU, one where its registers leave room for no more
    const int64_t heads = int64_t(c.B) * c.H;
    // More than 16 rows: in two workgroups, which both read the keys and values, where these fit on the card at once and a part is
    // short, so that what counts is latency (4 tokens and 8 heads, us in one / in two; D = 128: 8 sequences of 3000 22.2 / 21.9, 2 of 8000
    // 17.1 / 16.7; D = 256: 7 x 5 tokens of 6 heads in a window of 1024 20.8 / 17.6); in one where a part is long (16 of 5000 38.1 / 47.4,
    // 2 of 30000 26.8 / 32.7; D = 256: 1 of 20000 29.0 / 29.8) or there are more of them (40 of 3000: 54.7 / 62.6, D = 256 92.0 / 117.5).
    split_of(2 * heads, resident, kWaves, max_kv, &p.few_split, &p.few_each);
    if (p.few * c.G <= 16 || 2 * heads > resident || p.few_each > 16) {
      split_of(heads, resident, kWaves, max_kv, &p.few_split, &p.few_each);
      p.few_wide = p.few * c.G > 16 && 2 * heads * p.few_split > resident;
    }
    p.few_by_token = c.T <= int64_t(c.B) * p.few;
    room(p.few_by_token ? c.T : int64_t(c.B) * p.few, p.few_split, &p.few_o, &p.few_ml);
  }
  if (p.many) {
    // Tiles there can be: of T rows, with one broken tile a sequence.
    const auto tiles_of = [&](int64_t rows) { return std::min((most + rows - 1) / rows * c.B, c.T * c.G / rows + c.B) * c.H; };
    // The kernel of 256 rows a workgroup for long sequences whose work fills the card: each tile sees about as many positions, or
    // there are two tiles a CU (us with 128 rows a workgroup / with 256): 1024 x 8 rows on 30000 1056 / 863, 4 x 512 x 8 on 16000
    // 524 / 434, 256 x 4 on 8000 65 / 61; prompts, 8 heads of the cache, of 8192 x 4 545 / 485, 4096 x 4 162 / 137, 2048 x 8 91 / 82.
    // Fewer or shorter ones are better off with small tiles: prompts of 2048 x 4 60 / 66, of 4500 x 1 110 / 126, of 9000 x 1 224 / 234,
    // 8 of 1000 x 4 70 / 80, of 8192 x 4 with a window of 1024 180 / 185.
    const bool even = max_kv >= 2 * int64_t(c.max_new), full = tiles_of(2 * kTileRows) >= 512;
    p.tile_rows = c.D == 128 && max_kv >= 2048 && c.T * c.G >= 2 * kTileRows * int64_t(c.B) && (even || full) ? 2 * kTileRows : kTileRows;
    // Room for either kernel: which one it is goes by the window too, the workspace's size does not.
    const size_t from = at;
    size_t most_bytes = from;
    const auto plan = [&](int rows) {
      at = from;
      split_of(tiles_of(rows), rows > kTileRows || c.D > 128 ? 256 : 512, 8, max_kv, &p.many_split, &p.many_each);
      room(c.T, p.many_split, &p.many_o, &p.many_ml);
      most_bytes = std::max(most_bytes, at);
    };
    if (c.D == 128) plan(p.tile_rows == kTileRows ? 2 * kTileRows : kTileRows);
    p.many_o = p.many_ml = 0;
    plan(p.tile_rows);
    at = most_bytes;
  }
  p.ws_bytes = at;
  return p;
}

hipError_t launch_attention(const KvCall& call, const AttentionPlan& p, uint8_t* ws, hipStream_t s) {
  if (p.few) {
    KvCall c = call;
    c.lo_n = 1;
    c.hi_n = p.few;
    c.n_split = p.few_split;
    c.each = p.few_each;
    c.by_token = p.few_by_token;
    c.ws_o = reinterpret_cast<float*>(ws + p.few_o);
    c.ws_ml = reinterpret_cast<float*>(ws + p.few_ml);
    hipError_t e;
    switch (c.D) {
      case 64: e = pick<64>(c, p.few_wide, s); break;
      case 96: e = pick<96>(c, p.few_wide, s); break;
      case 128: e = pick<128>(c, p.few_wide, s); break;
      case 192: e = pick<192>(c, p.few_wide, s); break;
      default: e = pick<256>(c, p.few_wide, s);
    }
    if (e != hipSuccess) return e;
  }
  if (p.many) {
    KvCall c = call;
    c.lo_n = p.few + 1;
    c.hi_n = c.max_new;
    c.tile_rows = p.tile_rows;
    c.n_split = p.many_split;
    c.each = p.many_each;
    c.by_token = true;
    c.ws_o = reinterpret_cast<float*>(ws + p.many_o);
    c.ws_ml = reinterpret_cast<float*>(ws + p.many_ml);
    const hipError_t e = launch_attention_tiles(c, s);
    if (e != hipSuccess) return e;
    switch (c.D) {
      case 64: return join<64>(c, p.tile_rows, s);
      case 96: return join<96>(c, p.tile_rows, s);
      case 128: return join<128>(c, p.tile_rows, s);
      case 192: return join<192>(c, p.tile_rows, s);
      default: return join<256>(c, p.tile_rows, s);
    }
  }
  return hipSuccess;
}

}  // namespace hq
