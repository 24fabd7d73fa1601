// ep_moe_api.cpp -- the C ABI of the decode-side MoE operators (declared in
// include/ep_gb300_moe.h), with the conventions of ep_api.cpp: noexcept entry
// points, negative codes with a thread-local message, every configuration and
// argument checked on the host before anything is launched.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <exception>
#include <string>

#include "ep_cfg.hpp"
#include "ep_gb300_moe.h"
#include "ep_kernels.hpp"
#include "ep_moe_kernels.hpp"

using namespace epg;

namespace {

int fail(int code, const std::string& msg) { return RecordError(code, msg.c_str()); }

int fail_cuda(cudaError_t e, const char* what) {
  return fail(EP_ECUDA, std::string(what) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <class F>
int guarded(F&& f) noexcept {
  try {
    return f();
  } catch (const std::exception& ex) {
    return RecordError(EP_EINVAL, ex.what());
  } catch (...) {
    return RecordError(EP_EINVAL, "unknown exception");
  }
}

static_assert(EP_FEW_TOKENS == kFewTokens);

int check_route_cfg(const ep_route_cfg_t* c) {
  if (!c) return fail(EP_EINVAL, "route cfg is NULL");
  if (c->num_experts < 1 || c->num_experts > kMaxExperts)
    return fail(EP_EINVAL, "num_experts must be in [1, 2048]");
  if (c->topk < 1 || c->topk > kMaxTopk || c->topk > c->num_experts)
    return fail(EP_EINVAL, "topk must be in [1, min(16, num_experts)]");
  if (c->score != EP_SCORE_SOFTMAX && c->score != EP_SCORE_SIGMOID)
    return fail(EP_EINVAL, "score must be EP_SCORE_SOFTMAX or EP_SCORE_SIGMOID");
  if (c->renormalize != 0 && c->renormalize != 1) return fail(EP_EINVAL, "renormalize must be 0 or 1");
  if (!std::isfinite(c->scale)) return fail(EP_EINVAL, "scale must be finite");
  return EP_OK;
}

// The checks that ep_route and ep_route_backward share; fills p's common fields.
int check_logits(const ep_route_cfg_t* c, const void* logits, int32_t dtype, int64_t row_stride, int32_t n,
                 RouteParams* p) {
  if (const int rc = check_route_cfg(c); rc != EP_OK) return rc;
  if (n < 0 || n > kMaxTokens) return fail(EP_EINVAL, "num_tokens must be in [0, 2^24]");
  if (dtype != EP_BF16 && dtype != EP_FP32) return fail(EP_EINVAL, "logits must be EP_BF16 or EP_FP32");
  if (row_stride < c->num_experts) return fail(EP_EINVAL, "row_stride must be at least num_experts");
  if (n > 0) {
    if (!logits) return fail(EP_EINVAL, "logits is NULL");
    if (!aligned(logits, dtype == EP_BF16 ? 2 : 4)) return fail(EP_EINVAL, "logits must be aligned to its element");
  }
  p->logits = logits;
  p->row_stride = row_stride;
  p->n = n;
  p->experts = c->num_experts;
  p->topk = c->topk;
  p->bf16 = dtype == EP_BF16;
  p->sigmoid = c->score == EP_SCORE_SIGMOID;
  p->renorm = c->renormalize != 0;
  p->scale = c->scale;
  return EP_OK;
}

int check_route(const ep_route_cfg_t* cfg, const void* logits, int32_t dtype, int64_t row_stride,
                const float* select_bias, int32_t n, int64_t* idx, float* weights, RouteParams* p) {
  if (const int rc = check_logits(cfg, logits, dtype, row_stride, n, p); rc != EP_OK) return rc;
  if (n > 0) {
    if (!idx || !weights) return fail(EP_EINVAL, "topk_idx / topk_weights is NULL");
    if (!aligned(idx, 8) || !aligned(weights, 4) || !aligned(select_bias, 4))
      return fail(EP_EINVAL, "topk_idx, topk_weights and select_bias must be aligned to their elements");
  }
  p->bias = select_bias;
  p->idx = idx;
  p->weights = weights;
  return EP_OK;
}

bool group_ok(int32_t g) { return g == 32 || g == 64 || g == 128; }

int check_out(const void* out, int32_t dtype, uintptr_t align) {
  if (dtype != EP_BF16 && dtype != EP_FP32) return fail(EP_EINVAL, "out_dtype must be EP_BF16 or EP_FP32");
  if (out && !aligned(out, align ? align : (dtype == EP_BF16 ? 2u : 4u)))
    return fail(EP_EINVAL, "out is not aligned");
  return EP_OK;
}

int check_moe_cfg(const ep_moe_cfg_t* c) {
  if (!c) return fail(EP_EINVAL, "moe cfg is NULL");
  for (const int32_t d : {c->hidden_dim, c->intermediate_dim})
    if (d < 8 || d > kMaxHidden || d % 8 != 0)
      return fail(EP_EINVAL, "hidden_dim and intermediate_dim must be multiples of 8 in [8, 32768]");
  if (c->num_experts < 1 || c->num_experts > kMaxExperts)
    return fail(EP_EINVAL, "num_experts must be in [1, 2048]");
  if (c->num_expert_per_token < 1 || c->num_expert_per_token > kMaxTopk)
    return fail(EP_EINVAL, "num_expert_per_token must be in [1, 16]");
  if (c->max_tokens < 1 || c->max_tokens > EP_FEW_TOKENS)
    return fail(EP_EINVAL, "max_tokens must be in [1, 64]: larger batches go through ep_dispatch / ep_combine");
  if (c->activation != EP_ACT_SILU && c->activation != EP_ACT_GELU_TANH)
    return fail(EP_EINVAL, "activation must be EP_ACT_SILU or EP_ACT_GELU_TANH");
  if (c->weight_dtype == EP_INT4X2) {
    if (!group_ok(c->group_size)) return fail(EP_EINVAL, "group_size must be 32, 64 or 128");
    if (c->hidden_dim % c->group_size != 0 || c->intermediate_dim % c->group_size != 0)
      return fail(EP_EINVAL, "group_size must divide hidden_dim and intermediate_dim");
  } else if (c->weight_dtype == EP_BF16) {
    if (c->group_size != 0) return fail(EP_EINVAL, "group_size must be 0 with bf16 weights");
  } else {
    return fail(EP_EINVAL, "weight_dtype must be EP_BF16 or EP_INT4X2");
  }
  return EP_OK;
}

}  // namespace

struct ep_moe {
  ep_moe_cfg_t cfg{};
  int device = -1, num_sms = 0;
  cudaStream_t own_stream = nullptr;   // allocates, clears and frees the workspace
  cudaStream_t last_stream = nullptr;
  bool launched = false;
  void* block = nullptr;
  void* h = nullptr;
  float* part = nullptr;
  int32_t *ready = nullptr, *tile_done = nullptr, *blocks_done = nullptr, *err = nullptr;
  uint64_t wait_ns = 0;
};

namespace {

// What a block's warps may need of one another beside a wait for other blocks: microseconds.
constexpr uint64_t kBlockWaitNs = 2000000000ull;

// Checks of ep_moe_forward; fills the launch parameters.
int check_forward(ep_moe_t m, const void* x, int32_t n, const int64_t* idx, const float* w,
                  const ep_moe_weights_t* wt, const void* bias, void* out, int32_t out_dtype, MoeParams* p) {
  if (!m) return fail(EP_EINVAL, "handle is NULL");
  const ep_moe_cfg_t& c = m->cfg;
  if (n < 0 || n > c.max_tokens) return fail(EP_EINVAL, "num_tokens must be in [0, max_tokens]");
  if (const int rc = check_out(out, out_dtype, 16); rc != EP_OK) return rc;
  const bool int4 = c.weight_dtype == EP_INT4X2;
  if (n > 0) {
    if (!x || !idx || !w || !wt || !out) return fail(EP_EINVAL, "x, topk_idx, topk_weights, weights or out is NULL");
    if (!wt->w13 || !wt->w2) return fail(EP_EINVAL, "w13 / w2 is NULL");
    if (int4 != (wt->w13_scales != nullptr) || int4 != (wt->w2_scales != nullptr))
      return fail(EP_EINVAL, "4-bit weights need w13_scales and w2_scales, bf16 weights take none");
    if (!aligned(x, 16) || !aligned(bias, 16) || !aligned(wt->w13, 16) || !aligned(wt->w2, 16))
      return fail(EP_EINVAL, "x, bias, w13 and w2 must be 16-byte aligned");
    if (!aligned(idx, 8) || !aligned(w, 4) || !aligned(wt->w13_scales, 4) || !aligned(wt->w2_scales, 4))
      return fail(EP_EINVAL, "topk_idx, topk_weights and scales must be aligned to their elements");
    int dev = -1;
    if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
    if (dev != m->device)
      return fail(EP_EINVAL, "the current device is not the device the handle was created on");
    p->w13 = wt->w13;
    p->w13_scales = wt->w13_scales;
    p->w2 = wt->w2;
    p->w2_scales = wt->w2_scales;
  }
  p->x = x;
  p->topk_idx = idx;
  p->topk_weights = w;
  p->bias = bias;
  p->out = out;
  p->n = n;
  p->hidden = c.hidden_dim;
  p->inter = c.intermediate_dim;
  p->experts = c.num_experts;
  p->topk = c.num_expert_per_token;
  p->group = int4 ? c.group_size : 0;
  p->act = c.activation;
  p->out_f32 = out_dtype == EP_FP32;
  p->h = m->h;
  p->part = m->part;
  p->ready = m->ready;
  p->tile_done = m->tile_done;
  p->blocks_done = m->blocks_done;
  p->err = m->err;
  p->wait_ns = m->wait_ns;
  // A warp may wait for one that waits for another block, so that its limit has to be the
  // longer one; 0 gives up at the first test everywhere.
  p->block_wait_ns = m->wait_ns == 0 ? 0 : m->wait_ns + std::min(kBlockWaitNs, UINT64_MAX - m->wait_ns);
  return EP_OK;
}

int launch_moe(ep_moe_t m, const MoeParams& p, cudaStream_t s) {
  if (const cudaError_t e = LaunchMoe(p, m->num_sms, s); e != cudaSuccess) return fail_cuda(e, "MoE layer launch");
  m->last_stream = s;
  m->launched = true;
  return EP_OK;
}

}  // namespace

extern "C" {

int ep_route(const ep_route_cfg_t* cfg, const void* logits, int32_t logits_dtype, int64_t row_stride,
             const float* select_bias, int32_t num_tokens, int64_t* topk_idx, float* topk_weights,
             ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    RouteParams p{};
    if (const int rc = check_route(cfg, logits, logits_dtype, row_stride, select_bias, num_tokens, topk_idx,
                                   topk_weights, &p);
        rc != EP_OK)
      return rc;
    const cudaError_t e = LaunchRoute(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? EP_OK : fail_cuda(e, "route launch");
  });
}

int ep_route_backward(const ep_route_cfg_t* cfg, const void* logits, int32_t logits_dtype, int64_t row_stride,
                      const int64_t* topk_idx, const float* grad_weights, int32_t num_tokens, void* grad_logits,
                      int64_t grad_row_stride, ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    RouteParams p{};
    if (const int rc = check_logits(cfg, logits, logits_dtype, row_stride, num_tokens, &p); rc != EP_OK) return rc;
    if (grad_row_stride < cfg->num_experts) return fail(EP_EINVAL, "grad_row_stride must be at least num_experts");
    if (num_tokens > 0) {
      if (!topk_idx || !grad_weights || !grad_logits)
        return fail(EP_EINVAL, "topk_idx, grad_weights or grad_logits is NULL");
      if (!aligned(topk_idx, 8) || !aligned(grad_weights, 4) || !aligned(grad_logits, p.bf16 ? 2 : 4))
        return fail(EP_EINVAL, "topk_idx, grad_weights and grad_logits must be aligned to their elements");
    }
    p.idx_in = topk_idx;
    p.grad_w = grad_weights;
    p.grad = grad_logits;
    p.grad_stride = grad_row_stride;
    const cudaError_t e = LaunchRouteBackward(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? EP_OK : fail_cuda(e, "route backward launch");
  });
}

int ep_w4_linear(const void* x, int32_t num_tokens, const uint8_t* qweight, const float* scales, int32_t rows,
                 int32_t cols, int32_t group_size, void* out, int32_t out_dtype, ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    if (num_tokens < 0 || num_tokens > EP_FEW_TOKENS) return fail(EP_EINVAL, "num_tokens must be in [0, 64]");
    if (rows < 1 || rows > (1 << 24)) return fail(EP_EINVAL, "rows must be in [1, 2^24]");
    if (cols < 1 || cols > (1 << 18)) return fail(EP_EINVAL, "cols must be in [1, 2^18]");
    if (!group_ok(group_size)) return fail(EP_EINVAL, "group_size must be 32, 64 or 128");
    if (cols % group_size != 0) return fail(EP_EINVAL, "group_size must divide cols");
    if (const int rc = check_out(out, out_dtype, 0); rc != EP_OK) return rc;
    if (num_tokens > 0) {
      if (!x || !qweight || !scales || !out) return fail(EP_EINVAL, "x, qweight, scales or out is NULL");
      if (!aligned(x, 16) || !aligned(qweight, 16)) return fail(EP_EINVAL, "x and qweight must be 16-byte aligned");
      if (!aligned(scales, 4)) return fail(EP_EINVAL, "scales must be 4-byte aligned");
    }
    const W4Params p{x, qweight, scales, out, num_tokens, rows, cols, group_size, out_dtype == EP_FP32};
    const cudaError_t e = LaunchW4(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? EP_OK : fail_cuda(e, "4-bit product launch");
  });
}

int ep_moe_create(const ep_moe_cfg_t* cfg, ep_moe_t* out) noexcept {
  return guarded([&]() -> int {
    if (!out) return fail(EP_EINVAL, "out is NULL");
    *out = nullptr;
    if (const int rc = check_moe_cfg(cfg); rc != EP_OK) return rc;
    ep_moe* m = new ep_moe();
    m->cfg = *cfg;
    auto bail = [&](int code) {
      if (m->block) {
        cudaFreeAsync(m->block, m->own_stream);
        cudaStreamSynchronize(m->own_stream);
      }
      if (m->own_stream) cudaStreamDestroy(m->own_stream);
      delete m;
      return code;
    };
    cudaError_t e;
    if ((e = cudaGetDevice(&m->device)) != cudaSuccess) return bail(fail_cuda(e, "cudaGetDevice"));
    if ((e = cudaDeviceGetAttribute(&m->num_sms, cudaDevAttrMultiProcessorCount, m->device)) != cudaSuccess)
      return bail(fail_cuda(e, "cudaDeviceGetAttribute"));
    m->wait_ns = WaitLimitNs();
    const size_t entries = static_cast<size_t>(cfg->max_tokens) * cfg->num_expert_per_token;
    auto up = [](size_t b) { return (b + 255) & ~static_cast<size_t>(255); };
    const size_t n_h = up(entries * cfg->intermediate_dim * 6);
    const size_t n_part = up(entries * cfg->hidden_dim * sizeof(float));
    const size_t n_tile = static_cast<size_t>(cfg->hidden_dim + 15) / 16;
    const size_t total = n_h + n_part + up(sizeof(int32_t) * (cfg->num_experts + n_tile + 2));
    if ((e = cudaStreamCreateWithFlags(&m->own_stream, cudaStreamNonBlocking)) != cudaSuccess)
      return bail(fail_cuda(e, "cudaStreamCreateWithFlags"));
    if ((e = cudaMallocAsync(&m->block, total, m->own_stream)) != cudaSuccess) {
      cudaGetLastError();
      m->block = nullptr;
      return bail(fail(EP_ENOMEM, std::string("cudaMallocAsync of the layer's workspace failed: ") +
                                      cudaGetErrorString(e)));
    }
    char* b = static_cast<char*>(m->block);
    m->h = b;
    m->part = reinterpret_cast<float*>(b + n_h);
    m->ready = reinterpret_cast<int32_t*>(b + n_h + n_part);
    m->tile_done = m->ready + cfg->num_experts;
    m->blocks_done = m->tile_done + n_tile;
    m->err = m->blocks_done + 1;
    if ((e = cudaMemsetAsync(m->block, 0, total, m->own_stream)) != cudaSuccess)
      return bail(fail_cuda(e, "cudaMemsetAsync"));
    if ((e = cudaStreamSynchronize(m->own_stream)) != cudaSuccess)
      return bail(fail_cuda(e, "cudaStreamSynchronize"));
    *out = m;
    return EP_OK;
  });
}

int ep_moe_forward(ep_moe_t m, const void* x, int32_t num_tokens, const int64_t* topk_idx,
                   const float* topk_weights, const ep_moe_weights_t* weights, const void* bias, void* out,
                   int32_t out_dtype, ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    MoeParams p{};
    if (const int rc = check_forward(m, x, num_tokens, topk_idx, topk_weights, weights, bias, out, out_dtype, &p);
        rc != EP_OK)
      return rc;
    return launch_moe(m, p, reinterpret_cast<cudaStream_t>(stream));
  });
}

int ep_moe_layer(ep_moe_t m, const ep_route_cfg_t* route, const void* x, int32_t num_tokens, const void* logits,
                 int32_t logits_dtype, int64_t row_stride, const float* select_bias,
                 const ep_moe_weights_t* weights, const void* bias, int64_t* topk_idx, float* topk_weights,
                 void* out, int32_t out_dtype, ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    RouteParams r{};
    MoeParams p{};
    if (const int rc = check_route(route, logits, logits_dtype, row_stride, select_bias, num_tokens, topk_idx,
                                   topk_weights, &r);
        rc != EP_OK)
      return rc;
    if (const int rc = check_forward(m, x, num_tokens, topk_idx, topk_weights, weights, bias, out, out_dtype, &p);
        rc != EP_OK)
      return rc;
    if (route->num_experts != m->cfg.num_experts || route->topk != m->cfg.num_expert_per_token)
      return fail(EP_EINVAL, "the route cfg's num_experts and topk must be the handle's");
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (RoutesItself(r)) {   // one launch for the whole layer
      p.logits = r.logits;
      p.logits_stride = r.row_stride;
      p.idx_out = r.idx;
      p.weights_out = r.weights;
      p.route_scale = r.scale;
      p.logits_bf16 = r.bf16;
      p.sigmoid = r.sigmoid;
      p.renorm = r.renorm;
    } else if (const cudaError_t e = LaunchRoute(r, s); e != cudaSuccess) {
      return fail_cuda(e, "route launch");
    }
    return launch_moe(m, p, s);
  });
}

int ep_moe_status(ep_moe_t m, int32_t* device_error) noexcept {
  return guarded([&]() -> int {
    if (!m || !device_error) return fail(EP_EINVAL, "NULL argument");
    cudaStream_t s = m->launched ? m->last_stream : m->own_stream;
    int32_t v = 0;
    cudaError_t e = cudaMemcpyAsync(&v, m->err, sizeof v, cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return fail_cuda(e, "cudaMemcpyAsync");
    if ((e = cudaMemsetAsync(m->err, 0, sizeof v, s)) != cudaSuccess) return fail_cuda(e, "cudaMemsetAsync");
    if ((e = cudaStreamSynchronize(s)) != cudaSuccess) return fail_cuda(e, "cudaStreamSynchronize");
    *device_error = v;
    return EP_OK;
  });
}

void ep_moe_free(ep_moe_t m) noexcept {
  if (!m) return;
  if (m->launched) cudaStreamSynchronize(m->last_stream);
  if (m->block) {
    cudaFreeAsync(m->block, m->own_stream);
    cudaStreamSynchronize(m->own_stream);
  }
  if (m->own_stream) cudaStreamDestroy(m->own_stream);
  delete m;
}

}  // extern "C"
