// internal.h -- declarations shared by the C ABI (hq_api.cpp), the host prepack and the HIP
// launchers. Not part of the public interface.
#pragma once
#include <string>
#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "hq.h"
#include "layout.h"

namespace hq {

// A validated weight/activation/output combination.
struct Combo {
  Family fam;
  bool asym;     // WNA16 with zero-points
  bool out_i32;  // W8A8 raw accumulator output
  bool invariant;  // HQ_COMPUTE_BATCH_INVARIANT: one fixed kernel configuration for every M
  bool stream_k;   // HQ_COMPUTE_STREAM_K: small-M calls balanced over the CUs (Stream-K)
  int fine_group;  // decode calls only: INT4 weights with groups of 32 or 64 k (0: the format's own)
};

size_t prepacked_bytes(const Combo& c, int64_t E, int64_t N, int64_t K);
void prepack(const Combo& c, int64_t E, int64_t N, int64_t K, const void* wq, const void* scales,
             const void* zeros, void* out);

// The decode calls' layout (the format's own, or the fine-group one) and its prepack.
size_t decode_prepacked_bytes(const Combo& c, int64_t E, int64_t N, int64_t K);
void decode_prepack(const Combo& c, int64_t E, int64_t N, int64_t K, const void* wq, const void* scales,
                    const void* zeros, void* out);

// Kernel choice for one call (see dispatch in gemm_kernels.hip).
struct Plan {
  int kind;    // 0 = skinny (waves split K), 1 = tiled (LDS-staged activations), 2 = pipelined,
               // 3 = ping-pong, 4 = skinny Stream-K (one row block, `split` workgroups)
  int cfg;     // index into the kind's instantiation table
  int split;   // K splits across workgroups (partials in the workspace, then a reduction);
               // Stream-K: the number of workgroups
  size_t ws_bytes;
  long long sk_items = 0;   // Stream-K: (tile group, K unit) items
  int sk_slots = 0;         // Stream-K: partial-tile slots per tile group
};

struct GemmCall {
  Combo c;
  int64_t M, N, K;
  const void* a;
  const float* a_scale;
  const uint8_t* w;
  void* y;
  void* ws;
  size_t ws_bytes;
  hipStream_t stream;
  // MoE (sorted_ids != nullptr)
  const int32_t* sorted_ids;
  const int32_t* block_expert;
  const int32_t* num_padded;
  const float* topk_weights;
  int64_t T;
  int32_t topk;
  int32_t E;
  int32_t block_m;
  int64_t max_blocks;
};

Plan plan_dense(const Combo& c, int64_t M, int64_t N, int64_t K);
// Run-time tuning table (tuning_table.cpp): load (path NULL clears), lookup for a dense call.
int load_tuning_table(const char* path, std::string* err);
bool tuning_lookup(const Combo& c, int64_t M, int64_t N, int64_t K, int* kind, int* cfg, int* split);
int kernel_config_count(int kind);
Plan plan_moe(const Combo& c, int64_t T, int32_t topk, int32_t E, int64_t N, int64_t K,
              int32_t block_m);
int32_t moe_block_m(const Combo& c, int64_t T, int32_t topk, int32_t E, int64_t N, int64_t K);
bool moe_block_m_supported(int32_t block_m);
hipError_t launch_gemm(const GemmCall& call, const Plan& plan);
// hq_gemm_noalloc's workspace: a library-owned device array of kNoAllocScratchBytes per GPU; the
// device address of the current device's copy (looked up once per device).
constexpr size_t kNoAllocScratchBytes = size_t(HQ_NOALLOC_SCRATCH_BYTES);
hipError_t noalloc_scratch(void** ptr);

size_t moe_align_ws_bytes(int64_t T, int32_t topk, int32_t E, int32_t block_m);
hipError_t launch_grouped_index(const int32_t* offsets, int64_t R, int32_t E, int32_t bm, int64_t cap,
                                int32_t* sorted, int32_t* block_expert, int32_t* num_padded,
                                hipStream_t stream);
hipError_t launch_silu_mul(int64_t R, int64_t I, const void* gate_up, void* act, hipStream_t s);
hipError_t launch_moe_combine(int64_t T, int32_t topk, int32_t E, int64_t N, const int32_t* topk_ids,
                              const void* y, void* out, hipStream_t s);
hipError_t launch_act_quant(int act_fmt, int64_t M, int64_t K, const void* x, void* xq, float* s_tok,
                            hipStream_t stream);
hipError_t launch_silu_mul_quant(int act_fmt, int64_t R, int64_t I, const void* gate_up, void* act_q,
                                 float* act_scale, hipStream_t stream);

// hq_moe_route, validated.
struct RouteCall {
  const void* logits;
  const float* bias;
  int32_t* topk_ids;
  float* topk_weights;
  int64_t T;
  int E, topk, score_fn, bf16, n_group, topk_group, group_top, renormalize;
  float scale;
};
hipError_t launch_moe_route(const RouteCall& c, hipStream_t s);

// hq_gemv / hq_moe_decode, validated.
struct GemvCall {
  Combo c;
  bool gated;
  int64_t M, N, K;
  const void* x;
  const uint8_t* w;
  void* y;
};
hipError_t launch_gemv(const GemvCall& g, hipStream_t s);
struct DecW;
DecW dec_weights(const Combo& c, const uint8_t* w, int64_t N, int64_t K);
int dec_format(const Combo& c);
struct MoeDecodeCall {
  Combo c;
  int T, topk, E;
  int64_t H, I;
  const void* x;
  const int32_t* topk_ids;
  const float* topk_weights;
  const uint8_t* w_gate_up;
  const uint8_t* w_down;
  void* out;
  void* ws;
};
size_t moe_decode_ws_bytes(const Combo& c, int64_t T, int32_t topk, int32_t E, int64_t H, int64_t I);
hipError_t launch_moe_decode(const MoeDecodeCall& m, hipStream_t s);

// hq_rms_norm, validated.
struct RmsNormCall {
  int act_fmt;
  int64_t M, K;
  const void* x;
  const void* residual;
  const void* weight;
  float eps;
  void* residual_out;
  void* y;
  void* y_scale;
  void* y_bf16;
};
hipError_t launch_rms_norm(const RmsNormCall& a, hipStream_t s);

// hq_kv_append / hq_attention, validated.
struct KvCall {
  int fmt, H, D, page_shift, num_pages;   // the cache
  int B, max_new;
  int64_t T;
  const int32_t* cu;
  const int32_t* kv_lens;
  const int32_t* table;
  int width, capacity;                    // pages and positions of a sequence, at most
  uint32_t page_bytes;                    // codes of a page, all heads
  void* k_pages;
  void* v_pages;
  float* k_scales;
  float* v_scales;
  const void* k;                          // append
  const void* v;
  int64_t kv_stride;
  const void* q;                          // attention
  int64_t q_stride;
  int Hq, G, window;
  float scale_log2;                       // |sm_scale| * log2(e)
  uint32_t q_sign;                        // sm_scale < 0: the signs of two bf16
  void* out;
  int lo_n, hi_n;                         // one launch: sequences with that many new tokens,
  int tile_rows;                          // rows of a workgroup of the tiled kernels,
  int n_split, each;                      // parts of the positions at most, and blocks of a part at least,
  bool by_token;                          // partial results by row of q (else by sequence and token),
  float* ws_o;                            // averages [row][part][D], and (reference of the maximum, sum) of each part
  float* ws_ml;
};
hipError_t launch_kv_append(const KvCall& c, hipStream_t s);
int64_t attention_groups(const KvCall& c);   // workgroups without a split of the positions, at most
// Sequences of up to `few` new tokens have a launch of their own, those with more (many) another.
struct AttentionPlan {
  int few;
  bool many, few_by_token, few_wide;      // few_wide: 32 rows a workgroup, not 16
  int few_split, few_each, many_split, many_each, tile_rows;
  size_t few_o, few_ml, many_o, many_ml, ws_bytes;
};
AttentionPlan plan_attention(const KvCall& c, int64_t max_kv);
hipError_t launch_attention(const KvCall& c, const AttentionPlan& p, uint8_t* ws, hipStream_t s);
hipError_t launch_attention_tiles(const KvCall& c, hipStream_t s);

hipError_t launch_moe_align(const int32_t* topk_ids, int64_t T, int32_t topk, int32_t E,
                            int32_t block_m, int32_t* sorted_ids, int32_t* block_expert,
                            int32_t* expert_offsets, int32_t* num_padded, void* ws,
                            hipStream_t stream);

}  // namespace hq
