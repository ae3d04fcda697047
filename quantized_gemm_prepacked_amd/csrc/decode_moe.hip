// decode_moe.hip -- hq_moe_decode: the MoE layer for a few tokens in two launches.
//
//   up     act[t, j] = silu(Wg x[t]) * (Wu x[t]) for every routed entry (t, j)
//   down   out[t] = sum_j weight[t, j] * Wd act[t, j]
//
// Both stream expert weights through decode_ops.h. With few tokens an expert is hit by one or a few of
// them, so an expert's weights are read once for up to four of its tokens (a pass); more tokens on
// one expert take further passes, whose weights come from the caches.
// One token: a pass is a routed entry; ids outside [0, E) are left out. More: the up launch's first
// workgroups find an expert's tokens themselves (one lane per token looks through its own row of
// ids), and one extra workgroup writes the list of all passes that the down launch goes through.
//
// act stays between the launches as a high and a low bf16 (16 significant bits): the down product's A
// operand has unused MFMA rows, so the low half costs no matrix instruction, and the activations'
// rounding to 8 bits would otherwise be as large as the output's own.
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
};

__device__ __forceinline__ bool moe_valid(int e, int E) { return e >= 0 && e < E; }

// The list of passes (T > 1), by one workgroup: experts in the order of their first entry.
__device__ void moe_write_passes(const MoeParams& p, int32_t* ids, int32_t* count) {
  const int P = p.T * p.topk;
  for (int f = threadIdx.x; f < P; f += blockDim.x) ids[f] = p.ids[f];
  __syncthreads();
  // first entry of an expert: the number of its tokens' passes; elsewhere 0
  for (int f = threadIdx.x; f < P; f += blockDim.x) {
    const int e = ids[f];
    int passes = 0;
    if (moe_valid(e, p.E)) {
      bool first = true;
      for (int q = 0; q < f; ++q) first &= ids[q] != e;
      if (first) {
        int tokens = 0;
        for (int t = f / p.topk; t < p.T; ++t) {
          bool here = false;
          for (int j = 0; j < p.topk; ++j) here |= ids[t * p.topk + j] == e;
          tokens += here;
        }
        passes = (tokens + p.slots - 1) / p.slots;
      }
    }
    count[f] = passes;
  }
  __syncthreads();
  for (int f = threadIdx.x; f < P; f += blockDim.x) {
    if (count[f] == 0) continue;
    int at = 0;
    for (int q = 0; q < f; ++q) at += count[q];
    const int e = ids[f];
    int used = 0;
    Pass* s = p.passes + at;
    for (int t = f / p.topk; t < p.T; ++t) {
      int entry = -1;
      float w = 0.f;
      for (int j = 0; j < p.topk; ++j)
        if (ids[t * p.topk + j] == e) {
          if (entry < 0) entry = t * p.topk + j;
          w += p.weights ? p.weights[t * p.topk + j] : 1.0f;
        }
      if (entry < 0) continue;
      if (used == p.slots) {
        ++s;
        used = 0;
      }
      if (used == 0) {
        s->e = e;
        for (int g = 1; g < kSlots; ++g) {
          s->entry[g] = int16_t(entry);
          s->token[g] = -1;
        }
      }
      s->entry[used] = int16_t(entry);
      s->token[used] = int8_t(t);
      s->weight[used] = w;
      ++used;
    }
  }
  if (threadIdx.x == 0) {
    int total = 0;
    for (int q = 0; q < P; ++q) total += count[q];
    *p.n_passes = total;
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
  int f = blockIdx.y, e, slots = 1;
  uint32_t tokens = 0;   // bit t: token t is routed to e
  int entry = 0;         // AM = 4: lane t's first entry routed to e
  if constexpr (AM == 4) {
    if (f == 0) {
      if (blockIdx.x == 0) moe_write_passes(p, reinterpret_cast<int32_t*>(smem), reinterpret_cast<int32_t*>(smem) + p.T * p.topk);
      return;
    }
    --f;
    e = p.ids[f];
    if (!moe_valid(e, p.E)) return;
    entry = -1;
    if (lane < p.T)
      for (int j = p.topk - 1; j >= 0; --j)
        if (p.ids[lane * p.topk + j] == e) entry = lane * p.topk + j;
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
        [](int) __attribute__((always_inline)) {});

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

// NT tiles of 16 outputs per workgroup; the items (pass, K unit) are cut into NW equal contiguous
// ranges, one per wave. What a wave needs of an item -- its expert's address, its unit and pass, its
// activation rows -- is worked out 64 items at a time, one per lane, and read back by lane: done item
// by item on the scalar unit, which a CU's waves share, it took as long as the stream itself. AM = 2:
// one token, passes = its valid entries. AM = 6, 8: passes of up to two or four tokens, sums per token
// in LDS (a wave's own, so their order is the passes').
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
    count = __builtin_amdgcn_readfirstlane(*p.n_passes);
    const u32x4* from = reinterpret_cast<const u32x4*>(p.passes);
    for (int q = threadIdx.x; q < count * 2; q += NW * 64) reinterpret_cast<u32x4*>(passes)[q] = from[q];
    for (int q = threadIdx.x; q < NW * NT * p.T * 16; q += NW * 64) sums[q] = 0.f;
  }
  __syncthreads();

  const int out_tiles = p.N / 16, ot0 = blockIdx.x * NT, units = p.W.units;
  const int items = count * units;
  const int q0 = int(int64_t(items) * wave / NW), q1 = int(int64_t(items) * (wave + 1) / NW);
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
    dec_stream<F, AM, NT, D>(
        n, rows, rows_lds + wave * dec_wave_lds<AM, D>(), lane, acc,
        [&](int i) __attribute__((always_inline)) {
          const uint64_t lo = uint32_t(__builtin_amdgcn_readlane(w_lo, i)), hi = uint32_t(__builtin_amdgcn_readlane(w_hi, i));
          tile = dec_tile<F>(p.W, reinterpret_cast<const uint8_t*>(hi << 32 | lo), ot0, tiles);
          at = __builtin_amdgcn_readlane(u, i);
        },
        [&](int) __attribute__((always_inline)) { return tile; },
        // a tile past the last one lies outside the buffers
        [&](int, int t) __attribute__((always_inline)) { return at + t * units; },
        [&](int i, int r) __attribute__((always_inline)) { return row_at[i * RS + (r >> 1)] + (r & 1) * (p.K * 2); },
        [&](int i) __attribute__((always_inline)) {
          const int s = __builtin_amdgcn_readlane(du, i);
          if (s & 1) {
            const Pass& pass = passes[s >> 1];
            const int g = AM == 2 ? 0 : (lane >> 4) & (RS - 1);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              float v = dec_value<F, AM>(acc[t], 0) * pass.weight[g];
              if constexpr (DecTraits<F>::kW8) {
                const int c = min(ot0 + t, out_tiles - 1) * 16 + (lane & 15);
                const uint8_t* w = p.W.w + size_t(__builtin_amdgcn_readfirstlane(pass.e)) * p.W.expert_stride;
                v *= reinterpret_cast<const float*>(w + p.W.scales_off)[c];
              }
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
  const int T = AM == 2 ? 1 : p.T;
  for (int q = threadIdx.x; q < NT * T * 16; q += NW * 64) {
    const int c = q & 15, tok = (q >> 4) % T, t = (q >> 4) / T;
    if (ot0 + t >= out_tiles) continue;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) v += sums[((k * NT + t) * T + tok) * 16 + c];
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
  const int lds = std::max(std::max(red, rows), AM == 4 ? P * 8 : 0);
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
  const int tiles = p.N / 16;
  return launch(moe_down_kernel<F, AM, NT, NW, D>, dim3(unsigned((tiles + NT - 1) / NT)), NW * 64, lds, s, p);
}

// Workspace: the activations (high and low rows of every routed entry), the passes, their number.
struct MoeWs {
  size_t passes, count, total;
};
MoeWs moe_ws(int64_t T, int32_t topk, int64_t I) {
  MoeWs w;
  w.passes = align256(size_t(T) * topk * I * 4);
  w.count = w.passes + align256(size_t(T) * topk * sizeof(Pass));
  w.total = w.count + 256;
  return w;
}

template <int F>
hipError_t moe_fmt(const MoeDecodeCall& m, hipStream_t s) {
  const MoeWs ws = moe_ws(m.T, m.topk, m.I);
  uint8_t* base = static_cast<uint8_t*>(m.ws);
  uint16_t* act = reinterpret_cast<uint16_t*>(base);
  MoeParams up{dec_weights(m.c, m.w_gate_up, 2 * m.I, m.H), static_cast<const uint16_t*>(m.x), m.topk_ids, m.topk_weights, act,
               reinterpret_cast<Pass*>(base + ws.passes), reinterpret_cast<int*>(base + ws.count), m.T, m.topk, m.E,
               int(2 * m.I), int(m.H), m.T * m.topk > 2 * m.E ? 4 : 2};
  MoeParams down = up;
  down.W = dec_weights(m.c, m.w_down, m.H, m.I);
  down.x = act;
  down.y = static_cast<uint16_t*>(m.out);
  down.N = int(m.H);
  down.K = int(m.I);
  hipError_t e = m.T == 1 ? launch_up<F, 1, 1, 8, 2>(up, s) : launch_up<F, 4, 2, 4, 2>(up, s);
  if (e != hipSuccess) return e;
  if (m.T == 1) return m.H >= 6144 ? launch_down<F, 2, 2, 16, 2>(down, s) : launch_down<F, 2, 1, 16, 3>(down, s);
  if (up.slots == 4) return launch_down<F, 8, 1, 16, 2>(down, s);
  return m.H >= 6144 ? launch_down<F, 6, 2, 16, 2>(down, s) : launch_down<F, 6, 1, 16, 3>(down, s);
}

}  // namespace

size_t moe_decode_ws_bytes(const Combo&, int64_t T, int32_t topk, int32_t, int64_t, int64_t I) {
  return moe_ws(T, topk, I).total;
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
