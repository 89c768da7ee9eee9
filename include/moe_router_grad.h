/*
 * moe_router_grad.h -- what the router is trained with: the balance loss with
 * its per-expert counts, and the gradients from the layer's output back to
 * the router's weight and bias, C ABI.
 *
 * The experts are constants here (they may be the 4-bit ones of moe_q4.h):
 * no gradient of expert weights or of x is computed.  From the gradient of
 * the layer's output, the router's gradients take three calls:
 *   moe_finalize_backward     d_out, y       -> d_topk_w
 *   moe_route_backward        d_topk_w, loss -> d_logits
 *   moe_router_weight_grad    d_logits, x    -> d_wg, d_bias
 *
 * Conventions are those of moe_mi355x.h: device pointers to caller-owned,
 * 16-byte aligned, contiguous row-major memory; `stream` is a hipStream_t
 * passed as void*; host-side validation first, and on any error nothing is
 * enqueued and no output is touched.  Sums run in a fixed order: the same
 * call gives the same bits.  A workspace belongs to one call at a time: calls
 * that may overlap (other streams, other captured graphs) need their own.
 *
 * token_mask [T] uint8 or NULL: a token whose byte is 0 is padding.  It takes
 * no part in any count, mean or sum, its row of d_logits is exactly zero, and
 * its rows of logits, topk_ids, topk_w, d_topk_w and x may hold anything
 * (NaN, infinities, ids out of range).  NULL: every token is valid.
 * For the other tokens, logits, weights and gradients are finite, except
 * that a logit may be -infinity (an expert switched off: probability 0); a
 * row without any finite logit has probability 0 everywhere (moe_route gives no
 * finite weights for such a row: mask it, or pass weights of 0).  topk_ids and
 * topk_w are moe_route's: the k ids of a token are distinct and in [0, E) (an id
 * outside that range is skipped: nothing is read or written out of bounds,
 * and the result is then unspecified).
 */
#ifndef MOE_ROUTER_GRAD_H
#define MOE_ROUTER_GRAD_H

#include "moe_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes of moe_balance_loss for `shape`, or 0 if the shape is
 * invalid or unsupported.  Pure host function. */
size_t moe_balance_workspace_size(const moe_shape* shape);

/* Per-expert counts and the balance loss over the N valid tokens.
 *   p[t, :]      = softmax(logits[t, :]) over all E experts
 *   counts[e]    = routes of valid tokens to expert e         (int32 [E])
 *   mean_prob[e] = (1/N) sum_t p[t, e]                        (fp32 [E])
 *   loss         = E * sum_e counts[e] / (N k) * mean_prob[e] (fp32 [1])
 * 1 for a perfectly even router.  N == 0 (T == 0 too): all zero.
 * Probabilities in fp32, sums over tokens in fp64, one rounding.
 *   workspace: moe_balance_workspace_size(shape) bytes, 256-byte aligned. */
moe_status moe_balance_loss(const moe_shape* shape, const float* logits, const int32_t* topk_ids,
                            const uint8_t* token_mask, int32_t* counts, float* mean_prob,
                            float* loss, void* workspace, size_t workspace_bytes, void* stream);

/* Gradient with respect to the router logits of
 *   sum_tj d_topk_w[t, j] * topk_w[t, j]  +  d_loss[0] * balance loss,
 * where either part may be NULL (not both); the counts in the loss are
 * constants.  With f[e] = counts[e] / sum(counts), N = sum(counts) / k:
 *   balance part:  d_loss * E/N * p[t,e] * (f[e] - sum_e' f[e'] p[t,e'])
 *   weights part, renormalize = 1:  at e = topk_ids[t,j]
 *                  w[t,j] * (d_topk_w[t,j] - sum_i w[t,i] d_topk_w[t,i]), else 0
 *   weights part, renormalize = 0:
 *                  p[t,e] * ((d_topk_w[t,j] if e = topk_ids[t,j] else 0) - sum_i w[t,i] d_topk_w[t,i])
 *   topk_ids and topk_w are read only with d_topk_w, NULL is allowed without it.
 *   counts [E]: moe_balance_loss's for the same ids and mask; read only with
 *   d_loss, NULL is allowed without it.  d_loss [1] fp32 on the device.
 * Output d_logits [T, E] fp32 (every element written). */
moe_status moe_route_backward(const moe_shape* shape, const float* logits, const int32_t* topk_ids,
                              const float* topk_w, const uint8_t* token_mask, const int32_t* counts,
                              const float* d_topk_w, const float* d_loss, float* d_logits,
                              void* stream);

/* Workspace bytes of moe_router_weight_grad for `shape`, or 0 if the shape is
 * invalid or unsupported.  Pure host function. */
size_t moe_router_grad_workspace_size(const moe_shape* shape);

/* Gradients of the router's weight and bias:
 *   d_wg[e, h]  = sum over valid t of d_logits[t, e] * x[t, h]   (fp32 [E, H])
 *   d_bias[e]   = sum over valid t of d_logits[t, e]             (fp32 [E])
 * x [T, H] dtype; d_logits [T, E] fp32; d_bias may be NULL.  Products exact
 * to fp32 and better, sums in fp32.  T == 0: zeros are written.
 *   workspace: moe_router_grad_workspace_size(shape) bytes, 256-byte aligned. */
moe_status moe_router_weight_grad(const moe_shape* shape, const void* x, const float* d_logits,
                                  const uint8_t* token_mask, float* d_wg, float* d_bias,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of the routing weights, the backward pass of moe_finalize with
 * respect to topk_w:
 *   d_topk_w[t, j] = sum_n d_out[t, n] * y[inv[t*k + j], n]
 * y [R, H] as moe_grouped_gemm_down (or moe_q4_down) wrote it, inv
 * moe_permute's (values in [0, R), used unchecked), d_out [T, H] dtype.  The
 * small-token path of moe_forward and moe_forward_q4 leaves no y in the
 * workspace: run the down product on the workspace's h and offsets first.
 * Output d_topk_w [T, k] fp32; sums in fp32.  T == 0 enqueues nothing. */
moe_status moe_finalize_backward(const moe_shape* shape, const void* y, const int32_t* inv,
                                 const void* d_out, float* d_topk_w, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROUTER_GRAD_H */
