// moe_route.hip -- the router of an MoE layer: from a row of logits to the top-k experts and
// their weights, the step that makes the topk_ids / topk_weights every MoE call here takes.
//
// Per token: scores s = softmax(l) or sigmoid(l) over E experts, selection values v = s + bias,
// optionally only the best groups of experts kept, the k largest v in order (ties to the lowest
// id), weights from the scores s. One wave per token; the row's E <= 512 values live in registers,
// ceil(E / 64) per lane (expert i * 64 + lane, so the load is coalesced).
//
// Selection decides between neighbours, so it never compares rounded values: without a bias the
// order of s is the order of the logits themselves (both scores are strictly increasing), with a
// bias (or groups) s and v are held in 64 bits.
#include <hip/hip_runtime.h>

#include <cmath>

#include "device_ops.h"
#include "internal.h"

namespace hq {

namespace {

constexpr int kWaves = 4;   // tokens per workgroup

// The largest (v, lowest id) of the wave; every lane gets it.
__device__ __forceinline__ void wave_best(double& v, int& id) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const double ov = __shfl_xor(v, o);
    const int oi = __shfl_xor(id, o);
    if (ov > v || (ov == v && oi < id)) {
      v = ov;
      id = oi;
    }
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <int VPL, bool BF16>
__global__ __launch_bounds__(kWaves * 64) void moe_route_kernel(RouteCall c) {
  const int lane = threadIdx.x & 63;
  const int64_t t = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  if (t >= c.T) return;
  const double ninf = -__builtin_huge_val();

  // logits; NaN counts as -infinity, the value of a switched-off expert
  double l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 64 * i + lane;
    float f = -__builtin_huge_valf();
    if (e < c.E) {
      const size_t at = size_t(t) * c.E + e;
      f = BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(c.logits)[at]) : static_cast<const float*>(c.logits)[at];
      if (f != f) f = -__builtin_huge_valf();
    }
    l[i] = f;
  }

  double s[VPL], v[VPL];
  if (c.score_fn == HQ_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = 1.0 / (1.0 + exp(-l[i]));
  } else {
    double top = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = fmax(top, l[i]);
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmax(top, __shfl_xor(top, o));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      // equal to the maximum: 1 (also where both are infinite)
      s[i] = l[i] == ninf ? 0.0 : l[i] == top ? 1.0 : exp(l[i] - top);
      sum += s[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 64 * i + lane;
    double b = 0.0;
    if (c.bias && e < c.E) {
      b = c.bias[e];
      if (b != b) b = ninf;
    }
    v[i] = l[i] == ninf ? ninf : s[i] + b;
  }

  // groups: keep the experts of the best ones
  const int per = c.E / c.n_group;
  uint64_t kept = ~uint64_t(0);
  if (c.n_group > 1) {
    double mine = ninf;   // lane g < n_group: the value of group g
    for (int g = 0; g < c.n_group; ++g) {
      double sum = 0.0;
      int first = -1;
      bool any = false;
      for (int r = 0; r < c.group_top; ++r) {
        double bv = ninf;
        int bi = 1 << 30;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = 64 * i + lane;
          if (e < c.E && e / per == g && e != first && v[i] > bv) {
            bv = v[i];
            bi = e;
          }
        }
        wave_best(bv, bi);
        if (bv != ninf) {
          sum += bv;
          any = true;
        }
        first = bi;
      }
      if (lane == g && any) mine = sum;
    }
    kept = 0;
    for (int r = 0; r < c.topk_group; ++r) {
      double bv = mine;
      int bi = lane < c.n_group && !((kept >> lane) & 1) ? lane : 1 << 30;
      if (bi == 1 << 30) bv = ninf;
      wave_best(bv, bi);
      if (bi < 64) kept |= uint64_t(1) << bi;
    }
  }
  double by[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 64 * i + lane;
    const bool in = e < c.E && ((kept >> (c.n_group > 1 ? e / per : 0)) & 1) && v[i] != ninf;
    by[i] = !in ? ninf : c.bias ? v[i] : l[i];
  }

  // the k largest, one at a time; lane k keeps the k-th
  int my_id = -1;
  double my_s = 0.0, sum = 0.0;
  for (int k = 0; k < c.topk; ++k) {
    double bv = by[0];
    int bi = bv == ninf ? 1 << 30 : lane;
#pragma unroll
    for (int i = 1; i < VPL; ++i)
      if (by[i] > bv) {
        bv = by[i];
        bi = 64 * i + lane;
      }
    wave_best(bv, bi);
    if (bv == ninf) break;
    double sv = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (bi == 64 * i + lane) {
        sv = s[i];
        by[i] = ninf;
      }
    sv = __shfl(sv, bi & 63);
    sum += sv;
    if (lane == k) {
      my_id = bi;
      my_s = sv;
    }
  }
  if (lane < c.topk) {
    if (c.renormalize) my_s = sum > 0.0 ? my_s / sum : 0.0;
    c.topk_ids[t * c.topk + lane] = my_id;
    c.topk_weights[t * c.topk + lane] = float(my_s * c.scale);
  }
}

template <int VPL>
void launch(const RouteCall& c, dim3 grid, hipStream_t s) {
  if (c.bf16)
    hipLaunchKernelGGL((moe_route_kernel<VPL, true>), grid, dim3(kWaves * 64), 0, s, c);
  else
    hipLaunchKernelGGL((moe_route_kernel<VPL, false>), grid, dim3(kWaves * 64), 0, s, c);
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
