// ep_i8_api.cpp -- the C ABI of the int8 path (declared in include/ep_gb300_i8.h),
// with the conventions of ep_api.cpp.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "ep_api_checks.hpp"
#include "ep_cfg.hpp"
#include "ep_gb300_i8.h"
#include "ep_i8_kernels.hpp"

using namespace epg;
using namespace epg::api;

namespace {

int check_cols(int32_t cols) {
  if (cols < 16 || cols > EP_I8_MAX_COLS || cols % 16 != 0)
    return fail(EP_EINVAL, "cols must be a multiple of 16 in [16, 65536]");
  return EP_OK;
}

int check_x(const void* x, int32_t dtype, const int8_t* q, const float* scales) {
  if (!x || !q || !scales) return fail(EP_EINVAL, "x, q or scales is NULL");
  if (!aligned(x, dtype == EP_BF16 ? 2 : 4) || !aligned(scales, 4))
    return fail(EP_EINVAL, "x and scales must be aligned to their elements");
  if (!aligned(q, 16)) return fail(EP_EINVAL, "q must be 16-byte aligned");
  return EP_OK;
}

int check_x_dtype(int32_t dtype) {
  return dtype == EP_BF16 || dtype == EP_FP32 ? EP_OK : fail(EP_EINVAL, "x_dtype must be EP_BF16 or EP_FP32");
}

// The checks that both products share; fills p.  n: rows of x.
int check_product(const int8_t* x, const float* x_scales, int64_t n, const int8_t* w, const float* w_scales,
                  int32_t rows, int32_t cols, int32_t act, void* out, int32_t out_dtype, I8ProductParams* p) {
  if (rows < 1 || rows > (1 << 24)) return fail(EP_EINVAL, "rows must be in [1, 2^24]");
  if (const int rc = check_cols(cols); rc != EP_OK) return rc;
  if (act != EP_ACT_NONE && act != EP_ACT_SILU && act != EP_ACT_GELU_TANH)
    return fail(EP_EINVAL, "activation must be EP_ACT_NONE, EP_ACT_SILU or EP_ACT_GELU_TANH");
  if (act != EP_ACT_NONE && rows % 2 != 0) return fail(EP_EINVAL, "a gated product has an even number of rows");
  if (out_dtype != EP_BF16 && out_dtype != EP_FP32) return fail(EP_EINVAL, "out_dtype must be EP_BF16 or EP_FP32");
  if (n > 0) {
    if (!x || !x_scales || !w || !w_scales || !out) return fail(EP_EINVAL, "x, x_scales, w, w_scales or out is NULL");
    if (!aligned(x, 16) || !aligned(w, 16)) return fail(EP_EINVAL, "x and w must be 16-byte aligned");
    if (!aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(out, out_dtype == EP_BF16 ? 2 : 4))
      return fail(EP_EINVAL, "x_scales, w_scales and out must be aligned to their elements");
  }
  *p = {};
  p->x = x;
  p->x_scales = x_scales;
  p->w = w;
  p->w_scales = w_scales;
  p->out = out;
  p->n = n;
  p->rows = rows;
  p->cols = cols;
  p->act = act;
  p->out_f32 = out_dtype == EP_FP32;
  p->experts = 1;
  p->entries = n;
  p->wait_ns = WaitLimitNs();
  return EP_OK;
}

}  // namespace

extern "C" {

int ep_i8_quantize(ep_handle_t only_of, const void* x, int32_t x_dtype, int64_t row_stride, int64_t num_rows,
                   int32_t cols, int8_t* q, float* scales, ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    if (const int rc = check_x_dtype(x_dtype); rc != EP_OK) return rc;
    if (num_rows < 0 || num_rows > INT32_MAX) return fail(EP_EINVAL, "num_rows must be in [0, 2^31)");
    if (const int rc = check_cols(cols); rc != EP_OK) return rc;
    if (row_stride < cols) return fail(EP_EINVAL, "row_stride must be at least cols");
    if (num_rows > 0)
      if (const int rc = check_x(x, x_dtype, q, scales); rc != EP_OK) return rc;
    I8RowsParams p{};
    if (only_of) {
      Routing r;
      if (const int rc = RoutingOf(only_of, &r); rc != EP_OK) return rc;
      if (r.no_expand) return fail(EP_EINVAL, "only_of must be a handle of the expand layout");
      if (num_rows != r.rcap) return fail(EP_EINVAL, "num_rows must be the receive capacity of only_of");
      p.num_recv = r.num_recv;
      p.meta = r.meta;
      p.meta_stride = r.topk + 2;
    }
    p.x = x;
    p.row_stride = row_stride;
    p.rows = num_rows;
    p.cols = cols;
    p.bf16 = x_dtype == EP_BF16;
    p.q = q;
    p.scales = scales;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = LaunchI8Rows(p, s); e != cudaSuccess) return fail_cuda(e, "int8 rows launch");
    if (only_of) MarkUsed(only_of, s);
    return EP_OK;
  });
}

int ep_i8_dispatch(ep_handle_t h, const void* x, int32_t x_dtype, int8_t* recv_q, float* recv_scales,
                   ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    if (const int rc = check_x_dtype(x_dtype); rc != EP_OK) return rc;
    Routing r;
    if (const int rc = RoutingOf(h, &r); rc != EP_OK) return rc;
    if (const int rc = check_cols(r.hidden); rc != EP_OK) return fail(EP_EINVAL, "hidden_dim must be a multiple of 16");
    if (r.num_tokens > 0)
      if (const int rc = check_x(x, x_dtype, recv_q, recv_scales); rc != EP_OK) return rc;
    I8RowsParams p{};
    p.x = x;
    p.row_stride = r.hidden;
    p.rows = r.num_tokens;
    p.cols = r.hidden;
    p.bf16 = x_dtype == EP_BF16;
    p.q = recv_q;
    p.scales = recv_scales;
    p.slots = r.send_slot;
    p.topk = r.topk;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = LaunchI8Rows(p, s); e != cudaSuccess) return fail_cuda(e, "int8 dispatch launch");
    MarkUsed(h, s);
    return EP_OK;
  });
}

int ep_i8_linear(const int8_t* x, const float* x_scales, int32_t num_tokens, const int8_t* w, const float* w_scales,
                 int32_t rows, int32_t cols, int32_t activation, void* out, int32_t out_dtype,
                 ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    if (num_tokens < 0 || num_tokens > kMaxTokens) return fail(EP_EINVAL, "num_tokens must be in [0, 2^24]");
    I8ProductParams p;
    if (const int rc = check_product(x, x_scales, num_tokens, w, w_scales, rows, cols, activation, out, out_dtype, &p);
        rc != EP_OK)
      return rc;
    const cudaError_t e = LaunchI8Product(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? EP_OK : fail_cuda(e, "int8 product launch");
  });
}

int ep_i8_grouped(ep_handle_t h, const int8_t* x, const float* x_scales, const int8_t* w, const float* w_scales,
                  int32_t rows, int32_t cols, int32_t activation, void* out, int32_t out_dtype,
                  ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    Routing r;
    if (const int rc = RoutingOf(h, &r); rc != EP_OK) return rc;
    if (r.no_expand) return fail(EP_EINVAL, "the grouped product needs the expand layout");
    I8ProductParams p;
    // without tokens there is nothing to do, and no pointer is looked at
    if (const int rc = check_product(x, x_scales, r.num_tokens > 0 ? r.rcap : 0, w, w_scales, rows, cols, activation,
                                     out, out_dtype, &p);
        rc != EP_OK)
      return rc;
    // row numbers of tiles that reach past the end are 32 bits
    if (static_cast<int64_t>(r.experts) * rows > INT32_MAX - 4096 || r.rcap > INT32_MAX - 4096)
      return fail(EP_EINVAL, "experts * rows and the receive capacity must be below 2^31 - 4096");
    p.first = r.first;
    p.count = r.count;
    p.experts = r.experts;
    p.entries = static_cast<int64_t>(r.num_tokens) * r.topk;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (const cudaError_t e = LaunchI8Product(p, s); e != cudaSuccess) return fail_cuda(e, "grouped int8 product launch");
    MarkUsed(h, s);
    return EP_OK;
  });
}

int ep_i8_status(int32_t* device_error, ep_stream_t stream) noexcept {
  return guarded([&]() -> int {
    if (!device_error) return fail(EP_EINVAL, "device_error is NULL");
    const cudaError_t e = ReadI8Error(device_error, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? EP_OK : fail_cuda(e, "reading the int8 products' error word");
  });
}

}  // extern "C"
