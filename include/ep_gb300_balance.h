/*
 * ep_gb300_balance.h -- C ABI of the router's training losses in libep_gb300.so:
 * the load-balance loss and the z loss of a batch's router scores, the token
 * counts of the experts, and the gradient of the scores.
 *
 * The conventions are those of ep_gb300.h: device pointers of the current
 * device, work enqueued on `stream`, no synchronisation and no allocation in
 * the calls that do work (they can be captured into a CUDA graph), 0 or a
 * negative EP_E* code returned with a message from ep_last_error().
 */
#ifndef EP_GB300_BALANCE_H
#define EP_GB300_BALANCE_H

#include "ep_gb300_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque handle: the configuration and the workspace of the sums. */
typedef struct ep_balance *ep_balance_t;

/* Validate and allocate the workspace on the current device (stream-ordered on
 * a private stream, cleared, that stream alone waited for).  Of route the fields
 * num_experts (E), topk (K) and score are used; all have to be valid.
 * 1 <= max_tokens <= 2^24, 1 <= max_sequences <= 2^20. */
int ep_balance_create(const ep_route_cfg_t *route, int32_t max_tokens, int32_t max_sequences,
                      ep_balance_t *out) EP_NOEXCEPT;

/* Losses and counts.  logits: device bf16 or fp32 (logits_dtype) [num_tokens, E],
 * rows row_stride elements apart (row_stride >= E).  topk_idx: device int64
 * [num_tokens, K], what ep_route wrote; entries outside [0, E) count nowhere, and
 * a token whose K entries all are takes no part at all (padding, or a row with
 * every score masked).  The others are live.  seq_offsets: device int32 [G + 1],
 * ascending in [0, num_tokens]: sequence g has the tokens [seq_offsets[g],
 * seq_offsets[g + 1]); G = num_sequences.  NULL: one sequence of all tokens (G = 1).
 * Tokens outside every sequence take no part.  With z the logits in fp32 (-inf and
 * NaN are masked), per live token t
 *   p_te   = exp(z_te - lse_t)                  (EP_SCORE_SOFTMAX), or
 *            sigmoid(z_te) / sum_i sigmoid(z_ti)  (EP_SCORE_SIGMOID); 0 where masked
 *   lse_t  = log sum_e exp(z_te)                (both)
 * and
 *   tokens[g]       = T_g, the live tokens of g; tokens[G] = T, their sum     (int32 [G + 1])
 *   counts[g][e]    = entries of topk_idx of g's tokens that are e             (int32 [G, E])
 *   prob_sums[g][e] = sum of p_te over g's live tokens                        (fp32 [G, E])
 *   loss[0] = 1/G sum over g with T_g > 0 of E / (K T_g^2) sum_e counts[g][e] prob_sums[g][e]
 *   loss[1] = 1/T sum over the live tokens of lse_t^2                         (fp32 [2])
 * (loss[0] is 1 where every expert has its share; both are 0 without live tokens).
 * All scores of a live token masked: p is 0 and it adds nothing to loss[1].
 * Scores of +inf: p is that of the limit, loss[1] is inf.  Sums are fp32 in a fixed
 * order; equal inputs give equal bits on the same device.
 * 0 <= num_tokens <= max_tokens, 1 <= num_sequences <= max_sequences; every output
 * is written whole.  Offsets that are not ascending give unspecified sums. */
int ep_balance_forward(ep_balance_t b, const void *logits, int32_t logits_dtype, int64_t row_stride,
                       const int64_t *topk_idx, int32_t num_tokens, const int32_t *seq_offsets,
                       int32_t num_sequences, int32_t *counts, float *prob_sums, int32_t *tokens,
                       float *loss, ep_stream_t stream) EP_NOEXCEPT;

/* Gradient of the losses with respect to the logits (the counts are held fixed).
 * counts and tokens: what ep_balance_forward wrote for the same logits, topk_idx
 * and seq_offsets.  grad_loss: device fp32 [2], the incoming gradients of loss[0]
 * and loss[1] (the losses' coefficients, for a plain sum).  With c = counts[g],
 *   dz_j  = grad_loss[0] E / (G K T_g^2) p_j (c_j - sum_e c_e p_e) d_j
 *         + grad_loss[1] (2 / T) lse exp(z_j - lse)
 *   d_j   = 1 (softmax) or 1 - sigmoid(z_j) (sigmoid)
 * in fp32, 0 for masked scores and for tokens that are not live.  grad_logits:
 * device [num_tokens, E] of the logits' type, rows grad_row_stride elements apart:
 * accumulate 0: the value is stored; 1: it is added to what is there (in fp32, then
 * rounded), for example to the gradient that ep_route_backward wrote.  Rows
 * outside every sequence are left as they are.  grad_logits may not overlap logits. */
int ep_balance_backward(ep_balance_t b, const void *logits, int32_t logits_dtype, int64_t row_stride,
                        const int64_t *topk_idx, int32_t num_tokens, const int32_t *seq_offsets,
                        int32_t num_sequences, const int32_t *counts, const int32_t *tokens,
                        const float *grad_loss, void *grad_logits, int64_t grad_row_stride,
                        int32_t accumulate, ep_stream_t stream) EP_NOEXCEPT;

/* Release the handle; waits for the stream of its last call.  NULL is ignored.
 * One handle holds one workspace: order its forward calls (one stream, or events;
 * a captured graph counts as a call each time that it is replayed). */
void ep_balance_free(ep_balance_t b) EP_NOEXCEPT;

#ifdef __cplusplus
}
#endif

#endif /* EP_GB300_BALANCE_H */
