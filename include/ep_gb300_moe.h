/*
 * ep_gb300_moe.h -- C ABI of the decode-side MoE operators of libep_gb300.so:
 * the router (scores to top-k and its gradient), products with 4-bit weights,
 * and a whole MoE layer for a few tokens.
 *
 * The conventions are those of ep_gb300.h: device pointers of the current
 * device, work enqueued on `stream`, no synchronisation and no allocation in
 * the calls that do work (they can be captured into a CUDA graph), 0 or a
 * negative EP_E* code returned with a message from ep_last_error().  The
 * router's outputs are the topk_idx and topk_weights that ep_layout,
 * ep_dispatch_fwd and ep_combine take.
 */
#ifndef EP_GB300_MOE_H
#define EP_GB300_MOE_H

#include "ep_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ router */

enum { EP_SCORE_SOFTMAX = 0, EP_SCORE_SIGMOID = 1 };

/* Valid ranges: 1 <= num_experts <= 2048, 1 <= topk <= min(16, num_experts),
 * score one of EP_SCORE_*, renormalize 0 or 1, scale finite. */
typedef struct {
    int32_t num_experts;  /* E */
    int32_t topk;         /* K */
    int32_t score;        /* EP_SCORE_SOFTMAX or EP_SCORE_SIGMOID */
    int32_t renormalize;  /* 1: the K chosen scores are divided by their sum */
    float scale;          /* every weight is multiplied by it */
} ep_route_cfg_t;

/* Router: scores to top-k.  logits: device bf16 or fp32 (logits_dtype EP_BF16
 * or EP_FP32) [num_tokens, E], rows row_stride elements apart (row_stride >= E),
 * aligned to its element.  Per token t, with z_j the logits in fp32:
 *   f_j = exp(z_j - max) / sum_i exp(z_i - max)   (softmax)
 *   f_j = 1 / (1 + exp(-z_j))                     (sigmoid)
 *   S   = the K experts of largest z_j, or, with select_bias (device fp32 [E],
 *         may be NULL), of largest f_j + select_bias[j]; equal keys go to the
 *         lower id.  The bias takes part in the choice only.
 *   topk_idx[t][k]     = the k-th of S in that order (int64 [num_tokens, K])
 *   topk_weights[t][k] = scale * f_j / (renormalize ? sum of f over S : 1)
 *                        (fp32 [num_tokens, K])
 * A logit of -inf or NaN is masked: it takes no part in the sums and is never
 * chosen (neither is an expert whose biased key is NaN or -inf).  Where fewer
 * than K experts are left, the remaining entries are id -1 with weight 0 --
 * ep_layout's masked entry; a row with nothing left is all -1.  A +inf logit
 * ranks first; its softmax weight is that of the limit (the +inf logits share
 * the weight equally, the finite ones get 0).
 * 0 <= num_tokens <= 2^24. */
int ep_route(const ep_route_cfg_t *cfg, const void *logits, int32_t logits_dtype,
             int64_t row_stride, const float *select_bias, int32_t num_tokens,
             int64_t *topk_idx, float *topk_weights, ep_stream_t stream) EP_NOEXCEPT;

/* Gradient of ep_route's weights with respect to the logits (the choice of
 * experts is held fixed).  topk_idx: what ep_route wrote (a row's valid ids
 * are distinct; entries outside [0, E) are skipped and their gradient is not
 * read).  grad_weights: device fp32 [num_tokens, K].  grad_logits: device
 * [num_tokens, E] of the logits' type, rows grad_row_stride elements apart;
 * every element of the E columns is written.  With g_k the incoming gradient
 * times scale, f and S as above, a_k = f_k / sum over S of f:
 *   softmax, renormalised   dz_k = a_k (g_k - sum_S g a), 0 outside S
 *   softmax                 dz_j = f_j ([j in S] g_j - sum_S g f)
 *   sigmoid, renormalised   dz_k = a_k (g_k - sum_S g a) (1 - f_k), 0 outside S
 *   sigmoid                 dz_k = g_k f_k (1 - f_k), 0 outside S
 * computed in fp32, masked logits get 0.  grad_logits may not overlap logits. */
int ep_route_backward(const ep_route_cfg_t *cfg, const void *logits, int32_t logits_dtype,
                      int64_t row_stride, const int64_t *topk_idx, const float *grad_weights,
                      int32_t num_tokens, void *grad_logits, int64_t grad_row_stride,
                      ep_stream_t stream) EP_NOEXCEPT;

/* ----------------------------------------------------------- 4-bit weights */

/* The 4-bit form of a weight matrix W [rows, cols], symmetric with one fp32
 * scale per group of `group_size` consecutive columns of a row:
 *   qweight  uint8 [rows, cols/2]; byte b of a row holds column 2b in its low
 *            and column 2b+1 in its high nibble
 *   scales   fp32 [rows, cols/group_size]
 *   W[r][c] = (nibble - 8) * scales[r][c / group_size]
 * group_size is 32, 64 or 128 and divides cols; scales are below 2^122 in magnitude. */

/* Largest num_tokens of ep_w4_linear and largest max_tokens of ep_moe_create. */
#define EP_FEW_TOKENS 64

/* out[t][r] = sum_c W[r][c] * x[t][c].  x: device bf16 [num_tokens, cols];
 * out: device bf16 or fp32 (out_dtype) [num_tokens, rows].  Products of bf16
 * x and nibble - 8, each exact, are summed in fp32 per group, the groups'
 * sums times their scales in fp32; one rounding to bf16 at the end.
 * 0 <= num_tokens <= EP_FEW_TOKENS, 1 <= rows <= 2^24, 1 <= cols <= 2^18; x and
 * qweight 16-byte aligned, scales and out aligned to their elements. */
int ep_w4_linear(const void *x, int32_t num_tokens, const uint8_t *qweight, const float *scales,
                 int32_t rows, int32_t cols, int32_t group_size, void *out, int32_t out_dtype,
                 ep_stream_t stream) EP_NOEXCEPT;

/* --------------------------------------------- MoE layer for a few tokens */

/* weight_dtype of ep_moe_cfg_t: EP_BF16, or the 4-bit form above. */
enum { EP_INT4X2 = 4 };

enum { EP_ACT_SILU = 0, EP_ACT_GELU_TANH = 1 };

/* Valid ranges: hidden_dim and intermediate_dim multiples of 8 in [8, 32768]
 * (with EP_INT4X2 multiples of group_size), 1 <= num_experts <= 2048,
 * 1 <= num_expert_per_token <= 16, 1 <= max_tokens <= EP_FEW_TOKENS;
 * group_size 32, 64 or 128 with EP_INT4X2, else 0. */
typedef struct {
    int32_t hidden_dim;           /* H */
    int32_t intermediate_dim;     /* I */
    int32_t num_experts;          /* E */
    int32_t num_expert_per_token; /* K */
    int32_t max_tokens;           /* largest num_tokens of a call */
    int32_t weight_dtype;         /* EP_BF16 or EP_INT4X2 */
    int32_t group_size;           /* EP_INT4X2: columns per scale */
    int32_t activation;           /* EP_ACT_SILU or EP_ACT_GELU_TANH (of the gate) */
} ep_moe_cfg_t;

/* The experts' weights (device memory of the caller; only the experts that a
 * call's topk_idx names are read).
 *   w13  [E, 2*I, H]: rows 0..I-1 of an expert are the gate, I..2I-1 the up projection
 *   w2   [E, H, I]
 * each bf16, or qweight of the 4-bit form with its scales; 16-byte aligned
 * (scales 4-byte aligned, NULL for bf16). */
typedef struct {
    const void *w13;
    const float *w13_scales;
    const void *w2;
    const float *w2_scales;
} ep_moe_weights_t;

/* Opaque handle: the configuration and the workspace of the layer (the
 * intermediate activations and each expert row before the combine). */
typedef struct ep_moe *ep_moe_t;

/* Validate cfg and allocate the workspace on the current device (stream-ordered
 * on a private stream, cleared, that stream alone waited for). */
int ep_moe_create(const ep_moe_cfg_t *cfg, ep_moe_t *out) EP_NOEXCEPT;

/* The experts of a few tokens: for every token t
 *   h[t][k]  = act(W1[e] x[t]) * (W3[e] x[t]),  e = topk_idx[t][k], rounded to 16 significant bits
 *              (none of its 24 bits is dropped where out is fp32)
 *   out[t]   = sum over k ascending of topk_weights[t][k] * (W2[e] h[t][k])  (+ bias[t])
 * with fp32 sums; the expert rows W2 h stay fp32, the fold over k is the one
 * of ep_combine.  x: device bf16 [num_tokens, H]; topk_idx: device int64
 * [num_tokens, K]; topk_weights: device fp32 [num_tokens, K]; bias: device bf16
 * [num_tokens, H] or NULL; out: device bf16 or fp32 (out_dtype) [num_tokens, H],
 * may be bias itself when it has its type.  An entry of -1 is masked (its weight
 * is not read); any other id outside [0, E) is skipped and sets the value 1 in
 * the handle's error word.  A token with every entry masked gets 0 (+ bias).
 * 0 <= num_tokens <= max_tokens; x, bias and out 16-byte aligned.  Equal inputs
 * give equal bits: nothing depends on the order in which blocks run.  One
 * handle holds one workspace: order the calls on it (one stream, or events). */
int ep_moe_forward(ep_moe_t m, const void *x, int32_t num_tokens, const int64_t *topk_idx,
                   const float *topk_weights, const ep_moe_weights_t *weights, const void *bias,
                   void *out, int32_t out_dtype, ep_stream_t stream) EP_NOEXCEPT;

/* The whole layer: ep_route of logits [num_tokens, E] into topk_idx and
 * topk_weights (caller's buffers, as in ep_route), then ep_moe_forward with
 * them, to the same bits as those two calls.  route->num_experts and route->topk
 * must equal the handle's E and K.  One launch where the layer's kernel routes the
 * tokens itself (at most 8 tokens, 256 experts and 8 choices, no select_bias, and
 * not the softmax without renormalisation), else two. */
int ep_moe_layer(ep_moe_t m, const ep_route_cfg_t *route, const void *x, int32_t num_tokens,
                 const void *logits, int32_t logits_dtype, int64_t row_stride,
                 const float *select_bias, const ep_moe_weights_t *weights, const void *bias,
                 int64_t *topk_idx, float *topk_weights, void *out, int32_t out_dtype,
                 ep_stream_t stream) EP_NOEXCEPT;

/* Read and clear the handle's error word in order on the stream of its last
 * call, and wait for that stream only.  1 (bit 0): an expert id outside
 * [-1, E) was skipped; 2 (bit 1): a bounded device-side wait gave up
 * (EP_GB300_WAIT_NS when the handle was created; the call's output is then
 * not valid). */
int ep_moe_status(ep_moe_t m, int32_t *device_error) EP_NOEXCEPT;

/* Release the handle; waits for the stream of its last call.  NULL is ignored. */
void ep_moe_free(ep_moe_t m) EP_NOEXCEPT;

#ifdef __cplusplus
}
#endif

#endif /* EP_GB300_MOE_H */
