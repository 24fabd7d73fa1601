// ep_moe_kernels.hpp -- host-side interface between the C ABI of the decode-side
// MoE operators (ep_moe_api.cpp, include/ep_gb300_moe.h) and their kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace epg {

struct RouteParams {
  const void* logits;       // [n, E], rows row_stride elements apart
  const float* bias;        // [E] or null: added to the scores for the choice
  int64_t row_stride;
  int n, experts, topk;
  bool bf16, sigmoid, renorm;
  float scale;
  int64_t* idx;             // [n, K]
  float* weights;           // [n, K]
  // backward
  const int64_t* idx_in;    // [n, K]
  const float* grad_w;      // [n, K]
  void* grad;               // [n, E], rows grad_stride elements apart
  int64_t grad_stride;
};

cudaError_t LaunchRoute(const RouteParams& p, cudaStream_t s);
cudaError_t LaunchRouteBackward(const RouteParams& p, cudaStream_t s);

struct W4Params {
  const void* x;            // bf16 [n, cols]
  const uint8_t* q;         // [rows, cols/2]
  const float* scales;      // [rows, cols/group]
  void* out;                // [n, rows]
  int n, rows, cols, group;
  bool out_f32;
};

cudaError_t LaunchW4(const W4Params& p, cudaStream_t s);

constexpr int kFewTokens = 64;

struct MoeParams {
  const void* x;            // bf16 [n, H]
  const int64_t* topk_idx;  // [n, K]
  const float* topk_weights;
  // not null: the kernel routes the tokens itself (RoutesItself) and writes idx_out and weights_out
  const void* logits;       // [n, E], rows logits_stride elements apart
  int64_t logits_stride;
  int64_t* idx_out;         // [n, K]
  float* weights_out;       // [n, K]
  float route_scale;
  bool logits_bf16, sigmoid, renorm;
  const void* w13;          // [E, 2I, H]
  const float* w13_scales;
  const void* w2;           // [E, H, I]
  const float* w2_scales;
  const void* bias;         // bf16 [n, H] or null
  void* out;                // [n, H]
  int n, hidden, inter, experts, topk;
  int group;                // 0: bf16 weights
  int act;
  bool out_f32;
  // workspace
  void* h;                  // bf16 [max_tokens * K, 2 or (fp32 output) 3, I]: the parts that h is the sum of
  float* part;              // [max_tokens * K, H]
  // counters, zero between launches
  int32_t* ready;           // [E] finished gate/up rounds by expert
  int32_t* tile_done;       // [H / 16] finished down rounds by channel tile
  int32_t* blocks_done;     // [1]
  int32_t* err;
  uint64_t wait_ns;         // bound of one wait on other blocks
  uint64_t block_wait_ns;   // bound of one wait on other warps of the block
};

// Whether the MoE kernel can take this routing over: a warp a token, few experts and
// choices, weights that need no score but the chosen ones'.
constexpr int kOwnTokens = 8, kOwnExperts = 256, kOwnTopk = 8;
inline bool RoutesItself(const RouteParams& r) {
  return r.n <= kOwnTokens && r.experts <= kOwnExperts && r.topk <= kOwnTopk && r.bias == nullptr && (r.renorm || r.sigmoid);
}

cudaError_t LaunchMoe(const MoeParams& p, int num_sms, cudaStream_t s);

}  // namespace epg
