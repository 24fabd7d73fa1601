// ep_balance_api.cpp -- the C ABI of the router's training losses (declared in
// include/ep_gb300_balance.h), with the conventions of ep_api.cpp.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "ep_api_checks.hpp"
#include "ep_balance_kernels.hpp"
#include "ep_cfg.hpp"
#include "ep_gb300_balance.h"

using namespace epg;
using namespace epg::api;

struct ep_balance {
  ep_route_cfg_t cfg{};
  int max_tokens = 0, max_sequences = 0, device = -1, num_sms = 0;
  cudaStream_t own_stream = nullptr;   // allocates, clears and frees the workspace
  cudaStream_t last_stream = nullptr;
  bool launched = false;
  void* block = nullptr;
  float *sums = nullptr, *parts = nullptr;
  int32_t* ticket = nullptr;
};

namespace {

int check_cfg(const ep_route_cfg_t* c) {
  if (!c) return fail(EP_EINVAL, "route cfg is NULL");
  if (c->num_experts < 1 || c->num_experts > kMaxExperts) return fail(EP_EINVAL, "num_experts must be in [1, 2048]");
  if (c->topk < 1 || c->topk > kMaxTopk || c->topk > c->num_experts)
    return fail(EP_EINVAL, "topk must be in [1, min(16, num_experts)]");
  if (c->score != EP_SCORE_SOFTMAX && c->score != EP_SCORE_SIGMOID)
    return fail(EP_EINVAL, "score must be EP_SCORE_SOFTMAX or EP_SCORE_SIGMOID");
  if (c->renormalize != 0 && c->renormalize != 1) return fail(EP_EINVAL, "renormalize must be 0 or 1");
  if (!std::isfinite(c->scale)) return fail(EP_EINVAL, "scale must be finite");
  return EP_OK;
}

// The checks that both calls share; fills p's common fields.
int check_common(ep_balance_t b, const void* logits, int32_t dtype, int64_t row_stride, const int64_t* idx, int32_t n,
                 const int32_t* offsets, int32_t sequences, BalanceParams* p) {
  if (!b) return fail(EP_EINVAL, "handle is NULL");
  if (n < 0 || n > b->max_tokens) return fail(EP_EINVAL, "num_tokens must be in [0, max_tokens]");
  if (sequences < 1 || sequences > b->max_sequences)
    return fail(EP_EINVAL, "num_sequences must be in [1, max_sequences]");
  if (!offsets && sequences != 1) return fail(EP_EINVAL, "several sequences need seq_offsets");
  if (dtype != EP_BF16 && dtype != EP_FP32) return fail(EP_EINVAL, "logits must be EP_BF16 or EP_FP32");
  if (row_stride < b->cfg.num_experts) return fail(EP_EINVAL, "row_stride must be at least num_experts");
  if (!aligned(offsets, 4)) return fail(EP_EINVAL, "seq_offsets must be aligned to its element");
  if (n > 0) {
    if (!logits || !idx) return fail(EP_EINVAL, "logits / topk_idx is NULL");
    if (!aligned(logits, dtype == EP_BF16 ? 2 : 4) || !aligned(idx, 8))
      return fail(EP_EINVAL, "logits and topk_idx must be aligned to their elements");
  }
  int dev = -1;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
  if (dev != b->device) return fail(EP_EINVAL, "the current device is not the device the handle was created on");
  p->logits = logits;
  p->row_stride = row_stride;
  p->idx = idx;
  p->n = n;
  p->experts = b->cfg.num_experts;
  p->topk = b->cfg.topk;
  p->bf16 = dtype == EP_BF16;
  p->sigmoid = b->cfg.score == EP_SCORE_SIGMOID;
  p->offsets = offsets;
  p->sequences = sequences;
  p->sums = b->sums;
  p->parts = b->parts;
  p->ticket = b->ticket;
  p->num_sms = b->num_sms;
  p->blocks = BalanceBlocks(n, p->experts, b->num_sms);
  return EP_OK;
}

}  // namespace

extern "C" {

int ep_balance_create(const ep_route_cfg_t* route, int32_t max_tokens, int32_t max_sequences,
                      ep_balance_t* out) noexcept {
  return guarded([&]() -> int {
    if (!out) return fail(EP_EINVAL, "out is NULL");
    *out = nullptr;
    if (const int rc = check_cfg(route); rc != EP_OK) return rc;
    if (max_tokens < 1 || max_tokens > kMaxTokens) return fail(EP_EINVAL, "max_tokens must be in [1, 2^24]");
    if (max_sequences < 1 || max_sequences > (1 << 20)) return fail(EP_EINVAL, "max_sequences must be in [1, 2^20]");
    ep_balance* b = new ep_balance();
    b->cfg = *route;
    b->max_tokens = max_tokens;
    b->max_sequences = max_sequences;
    auto bail = [&](int code) {
      if (b->block) {
        cudaFreeAsync(b->block, b->own_stream);
        cudaStreamSynchronize(b->own_stream);
      }
      if (b->own_stream) cudaStreamDestroy(b->own_stream);
      delete b;
      return code;
    };
    cudaError_t e;
    if ((e = cudaGetDevice(&b->device)) != cudaSuccess) return bail(fail_cuda(e, "cudaGetDevice"));
    if ((e = cudaDeviceGetAttribute(&b->num_sms, cudaDevAttrMultiProcessorCount, b->device)) != cudaSuccess)
      return bail(fail_cuda(e, "cudaDeviceGetAttribute"));
    const size_t sums = BalanceSumWords(BalanceBlocks(max_tokens, route->num_experts, b->num_sms), max_sequences, route->num_experts);
    const size_t parts = BalancePartWords(max_sequences, route->num_experts);
    const size_t total = (sums + parts + 1) * sizeof(float);
    if ((e = cudaStreamCreateWithFlags(&b->own_stream, cudaStreamNonBlocking)) != cudaSuccess)
      return bail(fail_cuda(e, "cudaStreamCreateWithFlags"));
    if ((e = cudaMallocAsync(&b->block, total, b->own_stream)) != cudaSuccess) {
      cudaGetLastError();
      b->block = nullptr;
      return bail(fail(EP_ENOMEM, std::string("cudaMallocAsync of the losses' workspace failed: ") +
                                      cudaGetErrorString(e)));
    }
    b->sums = static_cast<float*>(b->block);
    b->parts = b->sums + sums;
    b->ticket = reinterpret_cast<int32_t*>(b->parts + parts);
    if ((e = cudaMemsetAsync(b->block, 0, total, b->own_stream)) != cudaSuccess)
      return bail(fail_cuda(e, "cudaMemsetAsync"));
    if ((e = cudaStreamSynchronize(b->own_stream)) != cudaSuccess)
      return bail(fail_cuda(e, "cudaStreamSynchronize"));
    *out = b;
    return EP_OK;
  });
}

int ep_balance_forward(ep_balance_t b, const void* logits, int32_t logits_dtype, int64_t row_stride,
                       const int64_t* topk_idx, int32_t num_tokens, const int32_t* seq_offsets, int32_t num_sequences,
                       int32_t* counts, float* prob_sums, int32_t* tokens, float* loss, ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    BalanceParams p{};
    if (const int rc = check_common(b, logits, logits_dtype, row_stride, topk_idx, num_tokens, seq_offsets,
                                    num_sequences, &p);
        rc != EP_OK)
      return rc;
    if (!counts || !prob_sums || !tokens || !loss)
      return fail(EP_EINVAL, "counts, prob_sums, tokens or loss is NULL");
    if (!aligned(counts, 4) || !aligned(prob_sums, 4) || !aligned(tokens, 4) || !aligned(loss, 4))
      return fail(EP_EINVAL, "counts, prob_sums, tokens and loss must be aligned to their elements");
    p.counts = counts;
    p.prob_sums = prob_sums;
    p.tokens = tokens;
    p.loss = loss;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = LaunchBalance(p, s); e != cudaSuccess) return fail_cuda(e, "balance launch");
    b->last_stream = s;
    b->launched = true;
    return EP_OK;
  });
}

int ep_balance_backward(ep_balance_t b, const void* logits, int32_t logits_dtype, int64_t row_stride,
                        const int64_t* topk_idx, int32_t num_tokens, const int32_t* seq_offsets,
                        int32_t num_sequences, const int32_t* counts, const int32_t* tokens, const float* grad_loss,
                        void* grad_logits, int64_t grad_row_stride, int32_t accumulate, ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    BalanceParams p{};
    if (const int rc = check_common(b, logits, logits_dtype, row_stride, topk_idx, num_tokens, seq_offsets,
                                    num_sequences, &p);
        rc != EP_OK)
      return rc;
    if (grad_row_stride < b->cfg.num_experts) return fail(EP_EINVAL, "grad_row_stride must be at least num_experts");
    if (accumulate != 0 && accumulate != 1) return fail(EP_EINVAL, "accumulate must be 0 or 1");
    if (num_tokens > 0) {
      if (!counts || !tokens || !grad_loss || !grad_logits)
        return fail(EP_EINVAL, "counts, tokens, grad_loss or grad_logits is NULL");
      if (!aligned(counts, 4) || !aligned(tokens, 4) || !aligned(grad_loss, 4) || !aligned(grad_logits, p.bf16 ? 2 : 4))
        return fail(EP_EINVAL, "counts, tokens, grad_loss and grad_logits must be aligned to their elements");
    }
    p.counts_in = counts;
    p.tokens_in = tokens;
    p.grad_loss = grad_loss;
    p.grad = grad_logits;
    p.grad_stride = grad_row_stride;
    p.accumulate = accumulate != 0;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = LaunchBalanceBackward(p, s); e != cudaSuccess) return fail_cuda(e, "balance backward launch");
    b->last_stream = s;
    b->launched = true;
    return EP_OK;
  });
}

void ep_balance_free(ep_balance_t b) noexcept {
  if (!b) return;
  if (b->launched) cudaStreamSynchronize(b->last_stream);
  if (b->block) {
    cudaFreeAsync(b->block, b->own_stream);
    cudaStreamSynchronize(b->own_stream);
  }
  if (b->own_stream) cudaStreamDestroy(b->own_stream);
  delete b;
}

}  // extern "C"
