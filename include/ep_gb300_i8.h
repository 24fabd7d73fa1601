/*
 * ep_gb300_i8.h -- C ABI of the 8-bit integer path of libep_gb300.so: rows to
 * int8 with one scale each (in place of their tokens, or dispatched to the receive
 * rows of a layout), and products of int8 rows with int8 weights, dense or
 * grouped by expert over the receive rows.
 *
 * The conventions are those of ep_gb300.h: device pointers of the current
 * device, work enqueued on `stream`, no synchronisation and no allocation in
 * the calls that do work (they can be captured into a CUDA graph), 0 or a
 * negative EP_E* code returned with a message from ep_last_error().  No output
 * may overlap an input.
 */
#ifndef EP_GB300_I8_H
#define EP_GB300_I8_H

#include "ep_gb300_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest cols of the calls here. */
#define EP_I8_MAX_COLS 65536

/* Rows to int8, symmetric with one fp32 scale a row.  x: device bf16 or fp32
 * (x_dtype) [num_rows, cols], rows row_stride elements apart (row_stride >= cols).
 *   scales[t] = max_c |x[t][c]| / 127                      (fp32 [num_rows])
 *   q[t][c]   = x[t][c] / scales[t], both in fp32, rounded to the nearest integer,
 *               ties to even, in [-127, 127]                (int8 [num_rows, cols])
 * scales[t] = 0 gives q = 0; a row that holds an infinity or a NaN gets scale NaN
 * and q = 0, so that every product with it is NaN.
 * only_of: NULL, or a handle of the expand layout (its cfg.no_expand 0): x has its
 * receive rows (num_rows is its receive capacity), and rows that receive nothing
 * are neither read nor written.
 * 0 <= num_rows < 2^31, cols a multiple of 16 in [16, EP_I8_MAX_COLS]; q 16-byte aligned, x and
 * scales aligned to their elements. */
int ep_i8_quantize(ep_handle_t only_of, const void *x, int32_t x_dtype, int64_t row_stride,
                   int64_t num_rows, int32_t cols, int8_t *q, float *scales,
                   ep_stream_t stream) EP_NOEXCEPT;

/* The int8 dispatch: x [N, H] (N the tokens of h's last ep_layout, H its
 * hidden_dim, a multiple of 16; contiguous rows) quantised as above, each row written to every
 * receive row of its token: recv_q int8 [Rcap, H], recv_scales fp32 [Rcap].
 * Rows that receive no token are not written.  Uses the routing of the last
 * ep_layout call, expand or not (its dispatch_dtype is not looked at). */
int ep_i8_dispatch(ep_handle_t h, const void *x, int32_t x_dtype, int8_t *recv_q, float *recv_scales,
                   ep_stream_t stream) EP_NOEXCEPT;

/* activation of the products: EP_ACT_* of ep_gb300_moe.h for a gated product, or */
enum { EP_ACT_NONE = -1 };

/* Product of int8 rows with int8 weights.  x: int8 [num_tokens, cols] and x_scales
 * fp32 [num_tokens] as above; w: int8 [rows, cols]; w_scales: fp32 [rows].
 *   y[t][r] = (sum_c w[r][c] x[t][c]) * w_scales[r] * x_scales[t]
 * with every product exact and sums in fp32 or int32 (whole numbers below 2^24
 * are exact in both); y in fp32.  EP_ACT_NONE: out[t][r] = y[t][r]
 * ([num_tokens, rows]).  EP_ACT_SILU, EP_ACT_GELU_TANH: the first rows / 2 rows
 * of w are the gate, the others the up projection (rows even), and
 *   out[t][r] = act(y[t][r]) * y[t][rows/2 + r]    ([num_tokens, rows / 2]).
 * out: device bf16 (one rounding at the end) or fp32 (out_dtype).
 * 0 <= num_tokens <= 2^24, 1 <= rows <= 2^24, cols a multiple of 16 in
 * [16, EP_I8_MAX_COLS]; x and w 16-byte aligned, the others aligned to their
 * elements.  Equal inputs give equal bits. */
int ep_i8_linear(const int8_t *x, const float *x_scales, int32_t num_tokens, const int8_t *w,
                 const float *w_scales, int32_t rows, int32_t cols, int32_t activation,
                 void *out, int32_t out_dtype, ep_stream_t stream) EP_NOEXCEPT;

/* The experts' products over the receive rows of h's last ep_layout (expand
 * layout; EP_EINVAL otherwise): receive row s of expert e, e's rows being the first
 * num_unaligned_recv_tokens_per_expert[e] from psum_num_recv_tokens_per_expert[e] on,
 *   out[s] = ep_i8_linear of x[s] with w[e] and w_scales[e].
 * x: int8 [Rcap, cols], x_scales: fp32 [Rcap]; w: int8 [E, rows, cols]; w_scales:
 * fp32 [E, rows]; out [Rcap, rows] (gated: [Rcap, rows / 2]).  cols and rows
 * need not be the handle's hidden_dim; E * rows and Rcap are below 2^31 - 4096.  Padding rows are left as they are, and what x
 * holds there does not matter. */
int ep_i8_grouped(ep_handle_t h, const int8_t *x, const float *x_scales, const int8_t *w,
                  const float *w_scales, int32_t rows, int32_t cols, int32_t activation,
                  void *out, int32_t out_dtype, ep_stream_t stream) EP_NOEXCEPT;

/* Read and clear the products' error word of the current device, in order on
 * `stream`, and wait for that stream only.  2 (bit 1): a bounded device-side wait
 * gave up (EP_GB300_WAIT_NS when the product was enqueued; the outputs of the products since
 * the last call of this are then not valid). */
int ep_i8_status(int32_t *device_error, ep_stream_t stream) EP_NOEXCEPT;

#ifdef __cplusplus
}
#endif

#endif /* EP_GB300_I8_H */
