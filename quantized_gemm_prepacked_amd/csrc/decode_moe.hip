// decode_moe.hip -- hq_moe_decode: the MoE layer for a few tokens in two launches.
//
//   up     act[t, j] = silu(Wg x[t]) * (Wu x[t]) for every routed entry (t, j)
//   down   out[t] = sum_j weight[t, j] * Wd act[t, j]
//
// Both stream expert weights through decode_ops.h, and reading them is what bounds them: at T = 1, 8 of
// 32 experts of 7168 x 2048 INT4, up reads 121 MB in 19.7 us (6.2 TB/s) and down 61 MB in 13.2 (4.6), where a kernel
// that only reads takes 19.4 and 10.9; at T = 16, 41 experts of 4096 x 1536 in groups of 32, 5.2 and 5.0 TB/s with
// the vector ALU 42 and 53 % busy. Below some 20 MB the two launches (2.3 us each) and their first loads' latency
// are most of it: 8 experts of 2048 x 768 MXFP4, 13.5 and 7.0 MB, take 6.2 and 5.6 us.
// With few tokens an expert is hit by one or a few of them, so its weights are read once for up to four
// of its tokens (a pass; in the down launch two, unless experts are shared widely); further tokens take
// further passes, whose weights come from the caches.
// One token: a pass is a routed entry; ids outside [0, E) are left out. More: the up launch's workgroups
// find an expert's tokens themselves (one lane per token looks through its own row of ids), and one extra
// workgroup writes the list of all passes that the down launch goes through.
//
// act stays between the launches as a high and a low bf16 (16 significant bits): the down product's A
// operand has unused MFMA rows, so the low half costs no matrix instruction, and the activations'
// rounding to 8 bits would otherwise be as large as the output's own (relative L2 against 64 bits 2.3e-3
// with it, 1.6e-3 without: the output's rounding alone).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "decode_ops.h"
#include "elementwise_ops.h"
#include "internal.h"

namespace hq {

namespace {

constexpr int kSlots = 4;   // tokens of a pass, at most

struct Pass {
  int e;                  // expert
  float weight[kSlots];   // router weight of a slot's token (an expert that stands in its row twice: the sum)
  int16_t entry[kSlots];  // the routed entry (t * topk + j) whose act row the slot reads
  int8_t token[kSlots];   // -1: no token (the slot repeats another's row and is dropped)
};
static_assert(sizeof(Pass) == 32 && HQ_MOE_DECODE_MAX_TOKENS * 64 <= 1 << 15, "Pass");

struct MoeParams {
  DecW W;
  const uint16_t* x;       // up: [T, H]; down: [entries][high, low][I]
  const int32_t* ids;
  const float* weights;
  uint16_t* y;             // up: act; down: out [T, H]
  Pass* passes;            // T > 1
  int* n_passes;
  int T, topk, E;
  int N, K;                // weight rows and K of this launch
  int slots;               // tokens of a pass of the down launch
  int tiles, splits;       // down: workgroups along the outputs, and along the items
  float* partial;          // splits > 1: [tiles][splits][the workgroup's sums]
  uint32_t* arrived;       // splits > 1: [tiles], zeroed by the up launch
};

__device__ __forceinline__ bool moe_valid(int e, int E) { return e >= 0 && e < E; }

// The list of passes (T > 1), by one workgroup of NW waves: experts in order, an expert's tokens in order,
// p.slots to a pass. lds: moe_pass_lds(P, E) bytes.
inline constexpr int moe_pass_lds(int P, int E) { return (P + 2 * E + 16) * 4; }

template <int NW>
__device__ void moe_write_passes(const MoeParams& p, uint8_t* lds) {
  const int P = p.T * p.topk, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int32_t* ids = reinterpret_cast<int32_t*>(lds);
  uint32_t* mask = reinterpret_cast<uint32_t*>(ids + P);   // bit t: token t is routed to the expert
  int32_t* base = reinterpret_cast<int32_t*>(mask + p.E);  // the expert's first pass
  int32_t* wave_sum = base + p.E;
  for (int e = tid; e < p.E; e += NW * 64) mask[e] = 0;
  for (int f = tid; f < P; f += NW * 64) ids[f] = p.ids[f];
  __syncthreads();
  for (int f = tid; f < P; f += NW * 64)
    if (moe_valid(ids[f], p.E)) atomicOr(&mask[ids[f]], 1u << (f / p.topk));
  __syncthreads();
  // exclusive prefix sum of the experts' passes, neighbouring experts per thread
  const int each = (p.E + NW * 64 - 1) / (NW * 64), e0 = tid * each;
  int mine = 0;
  for (int e = e0; e < min(e0 + each, p.E); ++e) mine += (__popc(mask[e]) + p.slots - 1) / p.slots;
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 63) wave_sum[wave] = upto;
  __syncthreads();
  int at = upto - mine;
  for (int w = 0; w < wave; ++w) at += wave_sum[w];
  for (int e = e0; e < min(e0 + each, p.E); ++e) {
    base[e] = at;
    at += (__popc(mask[e]) + p.slots - 1) / p.slots;
  }
  if (tid == NW * 64 - 1) *p.n_passes = at;
  __syncthreads();
  // each routed entry fills its token's slot; an expert's later entries in the same row only add their weight
  for (int f = tid; f < P; f += NW * 64) {
    const int e = ids[f], t = f / p.topk, row = t * p.topk;
    if (!moe_valid(e, p.E)) continue;
    bool again = false;
    for (int q = row; q < f; ++q) again |= ids[q] == e;
    if (again) continue;
    float w = 0.f;
    for (int q = f; q < row + p.topk; ++q)
      if (ids[q] == e) w += p.weights ? p.weights[q] : 1.0f;
    const uint32_t m = mask[e];
    const int r = __popc(m & ((1u << t) - 1)), g = r % p.slots;
    Pass* s = p.passes + base[e] + r / p.slots;
    if (g == 0) s->e = e;
    s->entry[g] = int16_t(f);
    s->token[g] = int8_t(t);
    s->weight[g] = w;
    if (r == __popc(m) - 1)   // the last token: the slots behind it repeat it
      for (int d = g + 1; d < p.slots; ++d) {
        s->entry[d] = int16_t(f);
        s->token[d] = -1;
      }
  }
}

// PAIRS pairs of (gate, up) tiles per workgroup; blockIdx.y: the routed entry (AM = 4: entry + 1, 0 the
// workgroup that lists the passes). An entry that is not the first of its expert leaves.
template <int F, int AM, int PAIRS, int NW, int D>
__global__ __launch_bounds__(NW * 64) void moe_up_kernel(MoeParams p) {
  constexpr int NT = 2 * PAIRS;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int I = p.N / 2;
  if (blockIdx.x == 0 && blockIdx.y == 0 && p.splits > 1)
    for (int q = threadIdx.x; q < p.tiles; q += NW * 64) p.arrived[q] = 0;
  int f = blockIdx.y, e, slots = 1;
  uint32_t tokens = 0;   // bit t: token t is routed to e
  int entry = 0;         // AM = 4: lane t's first entry routed to e
  if constexpr (AM == 4) {
    if (f == 0) {
      if (blockIdx.x == 0) moe_write_passes<NW>(p, smem);
      return;
    }
    --f;
    // lane t looks through token t's ids, eight loads at a time; the first eight are asked for together with
    // the entry's own
    const int32_t* row = p.ids + min(lane, p.T - 1) * p.topk;
    int32_t id[8];
    entry = -1;
    for (int j = 0; j < p.topk; j += 8) {
#pragma unroll
      for (int q = 0; q < 8; ++q) id[q] = row[min(j + q, p.topk - 1)];
      if (j == 0) {
        e = p.ids[f];
        if (!moe_valid(e, p.E)) return;
      }
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (id[q] == e && entry < 0) entry = min(j + q, p.topk - 1);
    }
    entry = entry >= 0 && lane < p.T ? lane * p.topk + entry : -1;
    tokens = uint32_t(__ballot(entry >= 0));
    if (__builtin_amdgcn_readlane(entry, __builtin_ctz(tokens)) != f) return;
    slots = __builtin_popcount(tokens);
  } else {
    e = p.ids[f];
    if (!moe_valid(e, p.E)) return;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  const uint8_t* w = p.W.w + size_t(e) * p.W.expert_stride;
  const int out_tiles = I / 16;
  const int ot0 = blockIdx.x * PAIRS;
  DecTile<F> tiles[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int ot = min(ot0 + t / 2, out_tiles - 1);
    tiles[t] = dec_tile<F>(p.W, w, t & 1 ? ot + out_tiles : ot);
  }
  const int n = p.W.units > wave ? (p.W.units - wave + NW - 1) / NW : 0;
  const rsrc_t rows = dec_rsrc(p.x, uint32_t(p.T) * p.K * 2);

  for (int s0 = 0; s0 < slots; s0 += AM) {
    // the pass's tokens (AM = 4), and their rows
    int tok[AM], ent[AM];
    if constexpr (AM == 4) {
#pragma unroll
      for (int g = 0; g < AM; ++g) {
        tok[g] = tokens ? __builtin_ctz(tokens) : tok[0];
        ent[g] = tokens ? __builtin_amdgcn_readlane(entry, tok[g]) : -1;
        tokens &= tokens - 1;
      }
    } else {
      tok[0] = 0;
      ent[0] = f;
    }
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    dec_stream<F, AM, NT, D>(
        n, rows, smem + wave * dec_wave_lds<AM, D>(), lane, acc,
        [](int) __attribute__((always_inline)) {}, [&](int t) __attribute__((always_inline)) { return tiles[t]; },
        [&](int i, int) __attribute__((always_inline)) { return wave + i * NW; },
        [&](int i, int r) __attribute__((always_inline)) {
          int t = tok[0];
          if constexpr (AM == 4) t = r == 0 ? tok[0] : r == 1 ? tok[1] : r == 2 ? tok[2] : tok[3];
          return uint32_t(t) * (p.K * 2) + uint32_t(wave + i * NW) * 256;
        },
        [](int, const DecUnit<F>(&)[NT]) __attribute__((always_inline)) {});

    float(*red)[NT][64] = reinterpret_cast<float(*)[NT][64]>(smem);
    __syncthreads();   // every wave is done with its activations
#pragma unroll
    for (int t = 0; t < NT; ++t) red[wave][t][lane] = dec_value<F, AM>(acc[t], 0);
    __syncthreads();
    for (int q = threadIdx.x; q < PAIRS * 64; q += NW * 64) {
      const int le = q & 63, o = q >> 6, g = le >> 4;
      int to = ent[0];
      if constexpr (AM == 4) to = g == 0 ? ent[0] : g == 1 ? ent[1] : g == 2 ? ent[2] : ent[3];
      if (g >= AM || to < 0 || ot0 + o >= out_tiles) continue;
      const int c = (ot0 + o) * 16 + (le & 15);
      float gate = 0.f, up = 0.f;
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        gate += red[v][2 * o][le];
        up += red[v][2 * o + 1][le];
      }
      if constexpr (DecTraits<F>::kW8) {
        const float* sc = reinterpret_cast<const float*>(w + p.W.scales_off);
        gate *= sc[c];
        up *= sc[c + I];
      }
      const float a = silu(gate) * up;
      const uint16_t hi = f32_to_bf16_rne(a);
      const float h = bf16_bits_to_f32(hi);
      // what the high half left out; nothing where it is infinite or NaN
      const uint16_t lo = fabsf(h) < __builtin_huge_valf() ? f32_to_bf16_rne(a - h) : uint16_t(0);
      uint16_t* act = p.y + size_t(to) * 2 * I + c;
      act[0] = hi;
      act[I] = lo;
    }
    __syncthreads();   // the sums are read before the next pass's rows land there
  }
}

// NT tiles of 16 outputs per workgroup; the items (pass, K unit) are cut into splits * NW equal contiguous
// ranges, one per wave of the splits workgroups (blockIdx.y) of a tile. With more than one, each leaves its
// sums in the workspace and the one that arrives last adds them, in split order.
// What a wave needs of an item -- its expert's address, its unit and pass, its activation rows -- is worked
// out 64 items at a time, one per lane, and read back by lane: done item by item on the scalar unit, which
// a CU's waves share, it took as long as the stream itself (T = 1, 7168 x 2048: 18.7 us against 17.8, and
// 2048 x 768: 6.5 against 5.3, tile shapes alike).
// AM = 2: one token, passes = its valid entries. AM = 6, 8: passes of up to two or four tokens, sums per
// token in LDS (a wave's own, so their order is the passes').
template <int F, int AM, int NT, int NW, int D>
__global__ __launch_bounds__(NW * 64) void moe_down_kernel(MoeParams p) {
  constexpr int RS = dec_rows<AM>() / 2;   // act rows (high and low) of an item
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int P = p.T * p.topk;
  Pass* passes = reinterpret_cast<Pass*>(smem);
  uint8_t* rows_lds = smem + P * sizeof(Pass);
  float* sums = reinterpret_cast<float*>(rows_lds + NW * dec_wave_lds<AM, D>());   // [NW][NT][T][16]
  int count;
  if constexpr (AM == 2) {
    const int e = lane < P ? p.ids[lane] : -1;
    const bool in = moe_valid(e, p.E);
    const uint64_t mask = __ballot(in);
    count = __popcll(mask);
    if (wave == 0 && in) {
      Pass& s = passes[__popcll(mask & ((uint64_t(1) << lane) - 1))];
      s.e = e;
      s.entry[0] = int16_t(lane);
      s.weight[0] = p.weights ? p.weights[lane] : 1.0f;
    }
  } else {
    // all P places, not the count's, so that the two loads do not wait for each other
    const u32x4* from = reinterpret_cast<const u32x4*>(p.passes);
    for (int q = threadIdx.x; q < P * 2; q += NW * 64) reinterpret_cast<u32x4*>(passes)[q] = from[q];
    count = __builtin_amdgcn_readfirstlane(*p.n_passes);
    for (int q = threadIdx.x; q < NW * NT * p.T * 16; q += NW * 64) sums[q] = 0.f;
  }
  __syncthreads();

  const int out_tiles = p.N / 16, ot0 = blockIdx.x * NT, units = p.W.units;
  const int items = count * units;
  const int part = blockIdx.y * NW + wave, parts = p.splits * NW;
  const int q0 = int(int64_t(items) * part / parts), q1 = int(int64_t(items) * (part + 1) / parts);
  f32x4 acc[NT];
  float total[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    total[t] = 0.f;
  }
  const int tiles = min(NT, out_tiles - ot0);
  const rsrc_t rows = dec_rsrc(p.x, uint32_t(P) * p.K * 4);
  uint32_t* row_at = reinterpret_cast<uint32_t*>(sums + NW * NT * p.T * 16) + wave * (64 * RS);
  for (int q = q0; q < q1; q += 64) {
    const int n = min(64, q1 - q);
    // lane i: item q + i
    const int qi = min(q + lane, q1 - 1);
    const int d = qi / units, u = qi - d * units;
    const uint64_t w_at = reinterpret_cast<uint64_t>(p.W.w) + uint64_t(passes[d].e) * p.W.expert_stride;
    const int w_lo = int(w_at), w_hi = int(w_at >> 32);
    const bool last = u == units - 1 || qi == q1 - 1;   // of this wave's units of the pass
    const int du = int(uint32_t(d) << 1 | uint32_t(last));
#pragma unroll
    for (int g = 0; g < RS; ++g) row_at[lane * RS + g] = uint32_t(passes[d].entry[g]) * (p.K * 4) + uint32_t(u) * 256;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // written by this wave, read by this wave

    DecTile<F> tile;
    int at = 0;
    dec_stream<F, AM, NT, D, true>(
        n, rows, rows_lds + wave * dec_wave_lds<AM, D>(), lane, acc,
        [&](int i) __attribute__((always_inline)) {
          const uint64_t lo = uint32_t(__builtin_amdgcn_readlane(w_lo, i)), hi = uint32_t(__builtin_amdgcn_readlane(w_hi, i));
          tile = dec_tile<F, true>(p.W, reinterpret_cast<const uint8_t*>(hi << 32 | lo), ot0, tiles);
          at = __builtin_amdgcn_readlane(u, i);
        },
        [&](int) __attribute__((always_inline)) { return tile; },
        // a tile past the last one lies outside the buffers
        [&](int, int t) __attribute__((always_inline)) { return at + t * units; },
        [&](int i, int r) __attribute__((always_inline)) { return row_at[i * RS + (r >> 1)] + (r & 1) * (p.K * 2); },
        [&](int i, const DecUnit<F>(&unit)[NT]) __attribute__((always_inline)) {
          const int s = __builtin_amdgcn_readlane(du, i);
          if (s & 1) {
            const Pass& pass = passes[s >> 1];
            const int g = AM == 2 ? 0 : (lane >> 4) & (RS - 1);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              float v = dec_value<F, AM>(acc[t], 0) * pass.weight[g];
              if constexpr (DecTraits<F>::kW8) v *= __uint_as_float(unit[t].s[0]);
              if constexpr (AM != 2) {
                const int tok = pass.token[g];
                if (tok >= 0 && (lane >> 4) < RS) sums[((wave * NT + t) * p.T + tok) * 16 + (lane & 15)] += v;
              } else {
                total[t] += v;
              }
              acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
          }
        });
  }

  if constexpr (AM == 2) {
    float(*red)[NT][16] = reinterpret_cast<float(*)[NT][16]>(sums);
    if (lane < 16) {
#pragma unroll
      for (int t = 0; t < NT; ++t) red[wave][t][lane] = total[t];
    }
  }
  __syncthreads();
  const int T = AM == 2 ? 1 : p.T, values = NT * T * 16;
  float* partial = p.partial + size_t(blockIdx.x) * p.splits * values;
  for (int q = threadIdx.x; q < values; q += NW * 64) {
    const int c = q & 15, tok = (q >> 4) % T, t = (q >> 4) / T;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) v += sums[((k * NT + t) * T + tok) * 16 + c];
    if (p.splits > 1)
      // device scope: written through to where every CU's loads see it
      __hip_atomic_store(partial + size_t(blockIdx.y) * values + q, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    else if (ot0 + t < out_tiles)
      p.y[size_t(tok) * p.N + (ot0 + t) * 16 + c] = f32_to_bf16_rne(v);
  }
  if (p.splits == 1) return;
  // every store above has completed before the workgroup counts as arrived; the last one's loads are of
  // device scope as well
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  int* last = reinterpret_cast<int*>(smem);
  if (threadIdx.x == 0)
    *last = __hip_atomic_fetch_add(p.arrived + blockIdx.x, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == uint32_t(p.splits);
  __syncthreads();
  if (!*last) return;
  for (int q = threadIdx.x; q < values; q += NW * 64) {
    const int c = q & 15, tok = (q >> 4) % T, t = (q >> 4) / T;
    if (ot0 + t >= out_tiles) continue;
    float v = 0.f;
    for (int k = 0; k < p.splits; ++k)
      v += __hip_atomic_load(partial + size_t(k) * values + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    p.y[size_t(tok) * p.N + (ot0 + t) * 16 + c] = f32_to_bf16_rne(v);
  }
}

template <class K>
hipError_t launch(K kern, dim3 grid, int threads, int lds, hipStream_t s, const MoeParams& p) {
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, grid, dim3(threads), lds, s, p);
  return hipGetLastError();
}

template <int F, int AM, int PAIRS, int NW, int D>
hipError_t launch_up(const MoeParams& p, hipStream_t s) {
  const int P = p.T * p.topk;
  constexpr int red = NW * 2 * PAIRS * 256, rows = NW * dec_wave_lds<AM, D>();
  const int lds = std::max(std::max(red, rows), AM == 4 ? moe_pass_lds(P, p.E) : 0);
  const int tiles = p.N / 32;
  return launch(moe_up_kernel<F, AM, PAIRS, NW, D>, dim3(unsigned((tiles + PAIRS - 1) / PAIRS), unsigned(P + (AM == 4 ? 1 : 0))),
                NW * 64, lds, s, p);
}

template <int F, int AM, int NT, int NW, int D>
hipError_t launch_down(const MoeParams& p, hipStream_t s) {
  const int P = p.T * p.topk;
  constexpr int rows = NW * (dec_wave_lds<AM, D>() + 64 * (dec_rows<AM>() / 2) * 4);
  // at most 1024 passes: 32 KiB of the 160
  static_assert(1024 * sizeof(Pass) + rows + NW * NT * (AM == 2 ? 1 : HQ_MOE_DECODE_MAX_TOKENS) * 64 <= 160 * 1024, "LDS");
  const int lds = P * int(sizeof(Pass)) + rows + NW * NT * p.T * 64;
  return launch(moe_down_kernel<F, AM, NT, NW, D>, dim3(unsigned(p.tiles), unsigned(p.splits)), NW * 64, lds, s, p);
}

// The down launch: tokens of a pass, tiles of a workgroup, workgroups along the outputs and the items.
struct DownPlan {
  int slots, nt, tiles, splits;
};
DownPlan down_plan(int64_t T, int32_t topk, int32_t E, int64_t H, int64_t I) {
  DownPlan d;
  d.slots = T * topk > 2 * E ? 4 : 2;
  d.nt = H >= 6144 && (T == 1 || d.slots == 2) ? 2 : 1;
  d.tiles = int((H / 16 + d.nt - 1) / d.nt);
  // Few output tiles leave CUs idle: then several workgroups share a tile's items, as long as a wave keeps
  // four units of distinct experts' weights (T = 16 top-8 of 128, 2048 x 768: 51 us as two, 57 as one; T = 4
  // top-2 of 16, 2048 x 1024: 13.1 as two, with two units a wave, 12.2 as one; T = 1 top-8 of 64, 1024 x 2048: 14.6
  // as three, 15.3 as two where a wave would have to keep eight).
  const int64_t units = std::min<int64_t>(T * topk, E) * (I / 128) / 16;
  d.splits = int(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(256 / d.tiles, units / 4), 16)));
  return d;
}

// Workspace: the activations (high and low rows of every routed entry), the passes, their number, the
// splits' sums and arrival counts.
struct MoeWs {
  size_t passes, count, partial, arrived, total;
};
MoeWs moe_ws(const DownPlan& d, int64_t T, int32_t topk, int64_t I) {
  MoeWs w;
  w.passes = align256(size_t(T) * topk * I * 4);
  w.count = w.passes + align256(size_t(T) * topk * sizeof(Pass));
  w.partial = w.count + 256;
  w.arrived = w.partial + (d.splits > 1 ? align256(size_t(d.tiles) * d.splits * d.nt * T * 64) : 0);
  w.total = w.arrived + (d.splits > 1 ? align256(size_t(d.tiles) * 4) : 0);
  return w;
}

// Tile shapes (tiles or pairs x waves x ring depth), us at the sizes of decode's benchmark cases:
//   up    T = 1: 1x8x2 20.4 at 7168 x 2048 and 5.5 at 2048 x 768 (1x8x4 21.7 / 5.8, 1x16x1 23.5 / 5.2);
//         T > 1: 2x4x2 20.4 at T = 3, 4096 x 1408 and 53 at T = 16, 4096 x 1536 (1x8x4 25.9 / 91: with eight
//         waves a wave has three or four units, and dead slots of the ring are a third of its loads)
//   down  T = 1: 2x16x2 13.4 at 7168 x 2048 but 6.9 at 2048 x 768, where half the CUs have no tile; 1x16x3
//         16.7 and 5.0 -- so two tiles a workgroup from H = 6144 on, where there are 192 workgroups (whole call,
//         I = 2048, one / two tiles: H = 4096 22.9 / 23.6, 5120 30.3 / 29.3, 6144 33.5 / 31.6; T = 3: 4096 43.1 /
//         43.2, 5120 55.3 / 52.5, 6144 63.5 / 59.0: from 257 tiles on two would do)
//         T > 1: 1x16x3 12.4 and 33 (2x16x2 16.3 / 48.6); with H = 7168 2x16x2 (T = 16 top-8 of 64: 253
//         against 269 for both launches); passes of four tokens where an expert has over two on average (T = 16
//         top-2 of 8, 4096 x 14336: 194 against 219 with passes of two)
template <int F>
hipError_t moe_fmt(const MoeDecodeCall& m, hipStream_t s) {
  const DownPlan d = down_plan(m.T, m.topk, m.E, m.H, m.I);
  const MoeWs ws = moe_ws(d, m.T, m.topk, m.I);
  uint8_t* base = static_cast<uint8_t*>(m.ws);
  uint16_t* act = reinterpret_cast<uint16_t*>(base);
  MoeParams up{};
  up.W = dec_weights(m.c, m.w_gate_up, 2 * m.I, m.H);
  up.x = static_cast<const uint16_t*>(m.x);
  up.ids = m.topk_ids;
  up.weights = m.topk_weights;
  up.y = act;
  up.passes = reinterpret_cast<Pass*>(base + ws.passes);
  up.n_passes = reinterpret_cast<int*>(base + ws.count);
  up.T = m.T;
  up.topk = m.topk;
  up.E = m.E;
  up.N = int(2 * m.I);
  up.K = int(m.H);
  up.slots = d.slots;
  up.tiles = d.tiles;
  up.splits = d.splits;
  up.partial = reinterpret_cast<float*>(base + ws.partial);
  up.arrived = reinterpret_cast<uint32_t*>(base + ws.arrived);
  MoeParams down = up;
  down.W = dec_weights(m.c, m.w_down, m.H, m.I);
  down.x = act;
  down.y = static_cast<uint16_t*>(m.out);
  down.N = int(m.H);
  down.K = int(m.I);
  const hipError_t e = m.T == 1 ? launch_up<F, 1, 1, 8, 2>(up, s) : launch_up<F, 4, 2, 4, 2>(up, s);
  if (e != hipSuccess) return e;
  if (m.T == 1) return d.nt == 2 ? launch_down<F, 2, 2, 16, 2>(down, s) : launch_down<F, 2, 1, 16, 3>(down, s);
  if (d.slots == 4) return launch_down<F, 8, 1, 16, 2>(down, s);
  return d.nt == 2 ? launch_down<F, 6, 2, 16, 2>(down, s) : launch_down<F, 6, 1, 16, 3>(down, s);
}

}  // namespace

size_t moe_decode_ws_bytes(const Combo&, int64_t T, int32_t topk, int32_t E, int64_t H, int64_t I) {
  return moe_ws(down_plan(T, topk, E, H, I), T, topk, I).total;
}

hipError_t launch_moe_decode(const MoeDecodeCall& m, hipStream_t s) {
  switch (dec_format(m.c)) {
    case DF_G128: return moe_fmt<DF_G128>(m, s);
    case DF_G128Z: return moe_fmt<DF_G128Z>(m, s);
    case DF_G64: return moe_fmt<DF_G64>(m, s);
    case DF_G64Z: return moe_fmt<DF_G64Z>(m, s);
    case DF_G32: return moe_fmt<DF_G32>(m, s);
    case DF_G32Z: return moe_fmt<DF_G32Z>(m, s);
    case DF_MXFP4: return moe_fmt<DF_MXFP4>(m, s);
    case DF_INT8: return moe_fmt<DF_INT8>(m, s);
    default: return moe_fmt<DF_FP8>(m, s);
  }
}

}  // namespace hq
