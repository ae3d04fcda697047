// moe_route.hip -- the router of an MoE layer: from a row of logits to the top-k experts and
// their weights, the step that makes the topk_ids / topk_weights every MoE call here takes.
//
// Per token: scores s = softmax(l) or sigmoid(l) over E experts, selection values v = s + bias,
// optionally only the best groups of experts kept, the k largest v in order (ties to the lowest
// id), weights from the scores s. One wave per token; the row's E <= 512 values live in registers,
// VPL = ceil(E / 64) neighbours per lane, so that among equal values the lowest lane, and in it the
// lowest place, is the lowest id.
//
// Selection decides between neighbours, so it never compares rounded values. Without bias and groups
// the order of s is the order of the logits themselves (both scores are strictly increasing): the keys are
// their 32 bits, and scores are worked out for the chosen ones only. Otherwise s and v are held in 64 bits.
//
// Bound by latency: one wave's chain of k wave-wide maxima, each six data-parallel moves inside the
// vector unit and one lane read (through LDS shuffles of 64-bit values and ids the same selection took
// twice as long).
#include <hip/hip_runtime.h>

#include <cmath>

#include "device_ops.h"
#include "internal.h"

namespace hq {

namespace {

constexpr int kWaves = 4;   // tokens per workgroup

// A lane's value moved within the wave (data-parallel primitive); lanes without a source get 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xF, false));
}

// Steps of a wave-wide fold into lane 63: shifts by 1, 2, 4, 8 inside rows of 16, then lane 15 of a row to
// the next one, then lane 31 to the upper half.
#define HQ_WAVE_FOLD(STEP) \
  STEP(0x111, 0xF) STEP(0x112, 0xF) STEP(0x114, 0xF) STEP(0x118, 0xF) STEP(0x142, 0xA) STEP(0x143, 0xC)

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define HQ_STEP(C, R) v = max(v, dpp<C, R>(v));
  HQ_WAVE_FOLD(HQ_STEP)
#undef HQ_STEP
  return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

__device__ __forceinline__ double make_f64(uint32_t hi, uint32_t lo) {
  return __longlong_as_double((long long)(uint64_t(hi) << 32 | lo));
}
__device__ __forceinline__ uint32_t hi32(double v) { return uint32_t(uint64_t(__double_as_longlong(v)) >> 32); }
__device__ __forceinline__ uint32_t lo32(double v) { return uint32_t(uint64_t(__double_as_longlong(v))); }

__device__ __forceinline__ double lane_f64(double v, int lane) {
  return make_f64(uint32_t(__builtin_amdgcn_readlane(int(hi32(v)), lane)), uint32_t(__builtin_amdgcn_readlane(int(lo32(v)), lane)));
}

// Sum over the wave, in a fixed order.
__device__ __forceinline__ double wave_sum(double v) {
#define HQ_STEP(C, R) v += make_f64(dpp<C, R>(hi32(v)), dpp<C, R>(lo32(v)));
  HQ_WAVE_FOLD(HQ_STEP)
#undef HQ_STEP
  return lane_f64(v, 63);
}

// Unsigned keys in the order of the values; 0 is below every key. Zeros must not be negative.
__device__ __forceinline__ uint32_t key_f32(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float f32_of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t key_f64(double f) {
  const uint64_t u = uint64_t(__double_as_longlong(f));
  return u ^ (uint64_t(int64_t(u) >> 63) | 0x8000000000000000ull);
}

// The largest value of the wave and the lowest lane that holds it.
__device__ __forceinline__ int best_lane(uint32_t key, uint32_t& best) {
  best = wave_max(key);
  return __builtin_ctzll(__ballot(key == best));
}
__device__ __forceinline__ int best_lane(uint64_t key, uint64_t& best) {
  const uint32_t hi = wave_max(uint32_t(key >> 32));
  const bool top = uint32_t(key >> 32) == hi;
  const uint32_t lo = wave_max(top ? uint32_t(key) : 0u);
  best = uint64_t(hi) << 32 | lo;
  return __builtin_ctzll(__ballot(key == best));
}

// exp(l - top), 1 where both are infinite.
__device__ __forceinline__ double exp_below(float l, float top) { return l == top ? 1.0 : exp(double(l) - double(top)); }
__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-double(l))); }

// PLAIN: no bias and no groups.
template <int VPL, bool BF16, bool PLAIN>
__global__ __launch_bounds__(kWaves * 64) void moe_route_kernel(RouteCall c) {
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int64_t t = int64_t(blockIdx.x) * kWaves + wave;
  const bool live = t < c.T;   // the workgroup's last waves may have no token; they take part in no barrier
  if (!live) return;
  const float ninf = -__builtin_huge_valf();
  const double ninf64 = -__builtin_huge_val();

  // logits; NaN counts as -infinity, the value of a switched-off expert; -0 as +0
  float l[VPL];
  uint32_t key[VPL];   // 0: switched off
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    float f = ninf;
    if (e < c.E) {
      const size_t at = size_t(t) * c.E + e;
      f = BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(c.logits)[at]) : static_cast<const float*>(c.logits)[at];
      f = f != f ? ninf : f + 0.0f;
    }
    l[i] = f;
    key[i] = f == ninf ? 0u : key_f32(f);
    most = max(most, key[i]);
  }
  const bool sigmoid = c.score_fn == HQ_SCORE_SIGMOID;

  int my_id = -1;      // lane k: the k-th choice
  double my_s = 0.0;   // and its score
  if constexpr (PLAIN) {
    uint32_t my_key = 0, first = 0;
    for (int k = 0; k < c.topk; ++k) {
      uint32_t m = key[0], best;
#pragma unroll
      for (int i = 1; i < VPL; ++i) m = max(m, key[i]);
      const int from = best_lane(m, best);
      if (best == 0) break;
      if (k == 0) first = best;
      int place = VPL - 1;
#pragma unroll
      for (int i = VPL - 2; i >= 0; --i) place = key[i] == best ? i : place;
      const int at = __builtin_amdgcn_readlane(place, from);
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = lane == from && i == at ? 0u : key[i];
      if (lane == k) {
        my_id = from * VPL + at;
        my_key = best;
      }
    }
    if (my_id >= 0) {
      const float mine = f32_of_key(my_key);
      my_s = sigmoid ? sigmoid64(mine) : exp_below(mine, f32_of_key(first));
    }
    if (!sigmoid && !c.renormalize) {   // renormalised, the sum over all experts cancels
      const float top = f32_of_key(first);
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += l[i] == ninf ? 0.0 : exp_below(l[i], top);
      sum = wave_sum(sum);
      my_s = sum > 0.0 ? my_s / sum : 0.0;
    }
  } else {
    __shared__ double group_v[kWaves][64 * VPL];
    double s[VPL], v[VPL];
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = l[i] == ninf ? 0.0 : sigmoid64(l[i]);
    } else {
      const float top = f32_of_key(wave_max(most));
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        s[i] = l[i] == ninf ? 0.0 : exp_below(l[i], top);
        sum += s[i];
      }
      sum = wave_sum(sum);
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      float b = 0.0f;
      if (c.bias && e < c.E) {
        b = c.bias[e];
        if (b != b) b = ninf;
      }
      v[i] = l[i] == ninf ? ninf64 : s[i] + double(b) + 0.0;
    }

    // groups: keep the experts of the best ones. LPG neighbouring lanes share a group (a power of two of
    // them), going through its values in the wave's own LDS, then fold their largest two.
    uint64_t kept = ~uint64_t(0);
    const int per = c.E / c.n_group;
    int lpg = 64;
    if (c.n_group > 1) {
      while (lpg * c.n_group > 64) lpg >>= 1;
      double* mine = group_v[wave];
#pragma unroll
      for (int i = 0; i < VPL; ++i) mine[lane * VPL + i] = v[i];
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // written and read by this wave alone
      const int g = lane / lpg;
      double a = ninf64, b = ninf64;   // the largest two
      if (g < c.n_group)
        for (int j = lane % lpg; j < per; j += lpg) {
          const double x = mine[g * per + j];
          b = fmax(b, fmin(a, x));
          a = fmax(a, x);
        }
      for (int o = 1; o < lpg; o <<= 1) {
        const double oa = __shfl_xor(a, o), ob = __shfl_xor(b, o);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      const double value = a == ninf64 ? ninf64 : (c.group_top == 2 && b != ninf64 ? a + b : a) + 0.0;
      // kept: fewer than topk_group groups are better (ties: the lower one is)
      int better = 0;
      for (int q = 0; q < c.n_group; ++q) {
        const double other = lane_f64(value, q * lpg);
        better += other > value || (other == value && q < g);
      }
      kept = __ballot(g < c.n_group && better < c.topk_group);   // bit lpg * g: group g
    }

    // the keys are the values' (bias) or still the logits' (groups alone)
    uint64_t by[VPL];
    int group = lane * VPL / per, in_group = lane * VPL - group * per;   // of the lane's next expert
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      const bool in = e < c.E && v[i] != ninf64 && ((kept >> (c.n_group > 1 ? group * lpg : 0)) & 1);
      if (++in_group == per) {
        in_group = 0;
        ++group;
      }
      by[i] = !in ? 0u : c.bias ? key_f64(v[i]) : uint64_t(key[i]);
    }
    for (int k = 0; k < c.topk; ++k) {
      uint64_t m = by[0], best;
#pragma unroll
      for (int i = 1; i < VPL; ++i) m = by[i] > m ? by[i] : m;
      const int from = best_lane(m, best);
      if (best == 0) break;
      int place = VPL - 1;
      double sv = s[VPL - 1];
#pragma unroll
      for (int i = VPL - 2; i >= 0; --i) {
        place = by[i] == best ? i : place;
        sv = by[i] == best ? s[i] : sv;
      }
      const int at = __builtin_amdgcn_readlane(place, from);
      sv = lane_f64(sv, from);
#pragma unroll
      for (int i = 0; i < VPL; ++i) by[i] = lane == from && i == at ? 0u : by[i];
      if (lane == k) {
        my_id = from * VPL + at;
        my_s = sv;
      }
    }
  }
  if (c.renormalize) {
    const double sum = wave_sum(my_s);   // lanes without a choice hold 0
    my_s = sum > 0.0 ? my_s / sum : 0.0;
  }
  if (lane < c.topk) {
    c.topk_ids[t * c.topk + lane] = my_id;
    c.topk_weights[t * c.topk + lane] = float(my_s * double(c.scale));
  }
}

template <int VPL>
void launch(const RouteCall& c, dim3 grid, hipStream_t s) {
  const bool plain = !c.bias && c.n_group == 1;
  const dim3 block(kWaves * 64);
  if (c.bf16) {
    if (plain) hipLaunchKernelGGL((moe_route_kernel<VPL, true, true>), grid, block, 0, s, c);
    else hipLaunchKernelGGL((moe_route_kernel<VPL, true, false>), grid, block, 0, s, c);
  } else {
    if (plain) hipLaunchKernelGGL((moe_route_kernel<VPL, false, true>), grid, block, 0, s, c);
    else hipLaunchKernelGGL((moe_route_kernel<VPL, false, false>), grid, block, 0, s, c);
  }
}

}  // namespace

hipError_t launch_moe_route(const RouteCall& c, hipStream_t s) {
  const dim3 grid(unsigned((c.T + kWaves - 1) / kWaves));
  if (c.E <= 64) launch<1>(c, grid, s);
  else if (c.E <= 128) launch<2>(c, grid, s);
  else if (c.E <= 256) launch<4>(c, grid, s);
  else launch<8>(c, grid, s);
  return hipGetLastError();
}

}  // namespace hq
