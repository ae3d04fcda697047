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
// twice as long). A lane's values are sorted once, so that a maximum looks at its first only and the
// winner moves up by one; of 64-bit keys the low halves are compared only where the high halves tie.
// Measured back to back (alone under a tracer): one row of 256 logits, top-8, 3.0 us (3.1), where a launch alone
// takes 2.2; 4096 rows with bias and 4 of 8 groups 10.4 us (11.3; its 4.5 MB would take 2.9), 8.6 without the groups
// and 8.1 with one choice instead of eight; without bias and groups, on 32-bit keys, 5.2.
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
  const uint64_t top = __ballot(uint32_t(key >> 32) == hi);
  int lane = __builtin_ctzll(top);
  uint32_t lo;
  if ((top & (top - 1)) == 0) {
    lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(key)), lane));
  } else {
    lo = wave_max(uint32_t(key >> 32) == hi ? uint32_t(key) : 0u);
    lane = __builtin_ctzll(__ballot(key == (uint64_t(hi) << 32 | lo)));
  }
  best = uint64_t(hi) << 32 | lo;
  return lane;
}

// A lane's keys in falling order with their places, equal ones in the order of their places (only
// neighbours are exchanged, and only where the later is larger).
template <int VPL, class K>
__device__ __forceinline__ void sort_keys(K (&key)[VPL], int (&place)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) place[i] = i;
#pragma unroll
  for (int n = VPL - 1; n > 0; --n)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool swap = key[i + 1] > key[i];
      const K a = key[i], b = key[i + 1];
      const int pa = place[i], pb = place[i + 1];
      key[i] = swap ? b : a;
      key[i + 1] = swap ? a : b;
      place[i] = swap ? pb : pa;
      place[i + 1] = swap ? pa : pb;
    }
}

// A lane's keys as one sorted list, or (eight of them, for which sorting costs more than it saves) two of
// the lower and the upper places.
template <int VPL, class K>
struct LaneKeys {
  static constexpr int kLists = VPL > 4 ? 2 : 1, kLen = VPL / kLists;
  K key[kLists][kLen];
  int place[kLists][kLen];
  __device__ __forceinline__ explicit LaneKeys(const K (&from)[VPL]) {
#pragma unroll
    for (int h = 0; h < kLists; ++h) {
#pragma unroll
      for (int i = 0; i < kLen; ++i) key[h][i] = from[h * kLen + i];
      sort_keys<kLen, K>(key[h], place[h]);
    }
  }
  __device__ __forceinline__ bool upper() const { return kLists == 2 && key[kLists - 1][0] > key[0][0]; }
  __device__ __forceinline__ K head() const { return upper() ? key[kLists - 1][0] : key[0][0]; }
  __device__ __forceinline__ int head_place() const { return upper() ? place[kLists - 1][0] + kLen : place[0][0]; }
  __device__ __forceinline__ void drop(bool yes) {
    const bool up = upper();
#pragma unroll
    for (int h = 0; h < kLists; ++h) {
      const bool mine = yes && up == (h == 1);
#pragma unroll
      for (int i = 0; i + 1 < kLen; ++i) {
        key[h][i] = mine ? key[h][i + 1] : key[h][i];
        place[h][i] = mine ? place[h][i + 1] : place[h][i];
      }
      key[h][kLen - 1] = mine ? K(0) : key[h][kLen - 1];
    }
  }
};

// The topk largest keys of the wave in order, keys of 0 left out: lane k gets the k-th one's id, -1 where
// there is none. first: the largest.
template <int VPL, class K>
__device__ __forceinline__ int choose(const K (&key)[VPL], int topk, int lane, K& first) {
  LaneKeys<VPL, K> keys(key);
  int id = -1;
  first = 0;
  for (int k = 0; k < topk; ++k) {
    K best;
    const int from = best_lane(keys.head(), best);
    if (best == 0) break;
    if (k == 0) first = best;
    const int at = __builtin_amdgcn_readlane(keys.head_place(), from);
    if (lane == k) id = from * VPL + at;
    keys.drop(lane == from);
  }
  return id;
}

// exp(l - top), 1 where both are +infinity, 0 at l = -infinity. (With nothing but switched-off logits top is
// NaN and so is every value: the sums are then not above 0, which gives weights of 0.)
__device__ __forceinline__ double exp_below(float l, float top) { return l == top ? 1.0 : exp(double(l) - double(top)); }
// From exp(-|l|), which cannot overflow: 1 / (1 + exp(-l)) would be 0 below -709.78, although the sigmoid is a
// number of binary64 down to -745, and a row of nothing but such logits still has weights.
__device__ __forceinline__ double sigmoid64(float l) {
  const double e = exp(-fabs(double(l)));
  return (l < 0.0f ? e : 1.0) / (1.0 + e);
}

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

  // logits; NaN counts as -infinity, the value of a switched-off expert; -0 as +0. Every lane loads (the
  // last expert again past the end), so that the loads stand together and are waited for once.
  float l[VPL];
  uint32_t key[VPL];   // 0: switched off
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const size_t at = size_t(t) * c.E + min(lane * VPL + i, c.E - 1);
    l[i] = BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(c.logits)[at]) : static_cast<const float*>(c.logits)[at];
  }
  float bias[VPL];
  if constexpr (!PLAIN) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) bias[i] = c.bias ? c.bias[min(lane * VPL + i, c.E - 1)] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    l[i] = lane * VPL + i >= c.E || l[i] != l[i] ? ninf : l[i] + 0.0f;
    key[i] = l[i] == ninf ? 0u : key_f32(l[i]);
    most = max(most, key[i]);
  }
  const bool sigmoid = c.score_fn == HQ_SCORE_SIGMOID;

  int my_id;           // lane k: the k-th choice, -1: none
  double my_s = 0.0;   // and its score
  if constexpr (PLAIN) {
    uint32_t first;
    my_id = choose<VPL>(key, c.topk, lane, first);
    // the chosen logits, from the lanes that hold them
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float x = __shfl(l[i], max(my_id, 0) / VPL);
      mine = my_id % VPL == i ? x : mine;
    }
    if (my_id >= 0) my_s = sigmoid ? sigmoid64(mine) : exp_below(mine, f32_of_key(first));
    if (!sigmoid && !c.renormalize) {   // renormalised, the sum over all experts cancels
      const float top = f32_of_key(first);
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += exp_below(l[i], top);
      sum = wave_sum(sum);
      my_s = sum > 0.0 ? my_s / sum : 0.0;
    }
  } else {
    __shared__ double group_v[kWaves][64 * VPL];
    double s[VPL], v[VPL];
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = sigmoid64(l[i]);   // 0 at -infinity
    } else {
      const float top = f32_of_key(wave_max(most));
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        s[i] = exp_below(l[i], top);
        sum += s[i];
      }
      sum = wave_sum(sum);
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float b = bias[i] != bias[i] ? ninf : bias[i];
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
    uint64_t first;
    my_id = choose<VPL>(by, c.topk, lane, first);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const double x = __shfl(s[i], max(my_id, 0) / VPL);
      if (my_id >= 0 && my_id % VPL == i) my_s = x;
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
