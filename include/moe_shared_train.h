/*
 * moe_shared_train.h -- the shared expert as a gated feed-forward block that
 * is trained, and dropout whose mask is stored nowhere, C ABI.
 *
 * moe_shared.h runs the shared expert for inference; here its forward pass
 * keeps what its backward pass reads, and the backward pass gives the
 * gradients of x and of both weights.  With the routed experts frozen, the
 * output's gradient d_out goes to moe_shared_ffn_backward as it is and, through
 * moe_finalize_backward (moe_router_grad.h), to the router.
 *
 * Conventions are those of moe_mi355x.h: device pointers to caller-owned,
 * 16-byte aligned, contiguous row-major memory; `stream` is a hipStream_t
 * passed as void*; host-side validation first, and on any error nothing is
 * enqueued and no output is touched.  Of `shape`, T, H and dtype matter here
 * (all fields are checked).  An output overlaps no input and no other output,
 * except where it says so.  Sums run in a fixed order: the same call gives the
 * same bits.  A workspace belongs to one call at a time: calls that may
 * overlap (other streams, other captured graphs) need their own.
 *
 * Envelope, beside moe_mi355x.h's: Is % 32 == 0, 2*T*Is < 2^31, w1s below
 * 4 GiB, H and 2*Is at most 2^20; otherwise MOE_ERR_UNSUPPORTED.  Is <= 0 is
 * MOE_ERR_INVALID_ARG.
 *
 * Dropout.  rng: two uint64 on the device, seed and offset (NULL is allowed
 * where p rounds to 0).  They are read by the kernels, so a captured graph that
 * is replayed takes what they hold then; a backward call needs the values its
 * forward call had.  Calls whose masks must differ need another seed or offset.
 * An element e of a tensor (its row-major index) is dropped where
 *   u16(e) < cut,  cut = floor(p * 65536 + 1/2);  else it is scaled by 65536 / (65536 - cut),
 * u16(e) being bits 16*(e%8) .. of the 128-bit block that Philox 4x32 with ten
 * rounds (Salmon, Moraes, Dror, Shaw, SC 2011) makes of the counter words
 * (e/8 low, e/8 high, offset low, offset high) under the key (seed low, seed
 * high).  A dropped element is 0 whatever its value was.  p outside [0, 1), or
 * so near 1 that cut is 65536, is MOE_ERR_INVALID_ARG.
 */
#ifndef MOE_SHARED_TRAIN_H
#define MOE_SHARED_TRAIN_H

#include "moe_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/* out = residual + dropout(y), all [T, H] dtype, one rounding; residual may be
 * NULL (none).  out may be y or residual.  T == 0 enqueues nothing. */
moe_status moe_dropout_add(const moe_shape* shape, double p, const uint64_t* rng, const void* y,
                           const void* residual, void* out, void* stream);

/* Gradient of y: d_y = dropout(d_out) with the forward call's mask.  (The
 * residual's gradient is d_out.)  d_y may be d_out. */
moe_status moe_dropout_backward(const moe_shape* shape, double p, const uint64_t* rng,
                                const void* d_out, void* d_y, void* stream);

/* Forward pass:
 *   gu[t, i]  = x[t] . w1s[i]                                    (i < 2*Is: gate, then up)
 *   hs[t, i]  = dropout(SiLU(gate[t, i]) * up[t, i])             (its index t*Is + i)
 *   out[t, n] = sum_i hs[t, i] * w2s[n, i] + residual[t, n]
 * x, out [T, H], w1s [2*Is, H], w2s [H, Is] as in moe_shared.h; gu [T, 2*Is]
 * (fp32) and hs [T, Is] are kept for the backward pass; hs and out in dtype,
 * each rounded once.  residual [T, H] may be NULL; out
 * may be residual.  T == 0 enqueues nothing. */
moe_status moe_shared_ffn_train(const moe_shape* shape, int32_t Is, double p, const uint64_t* rng,
                                const void* x, const void* w1s, const void* w2s,
                                const void* residual, float* gu, void* hs, void* out, void* stream);

/* Workspace bytes of moe_shared_ffn_backward, or 0 if shape or Is is invalid
 * or unsupported.  Pure host function. */
size_t moe_shared_backward_workspace_size(const moe_shape* shape, int32_t Is);

/* Backward pass from d_out [T, H], with x, the weights, gu and hs of the
 * forward call and its p and rng values:
 *   dh     = dropout(d_out w2s)
 *   dg, du = dh * up * s * (1 + gate * (1 - s)),  dh * gate * s,   s = 1 / (1 + e^-gate)
 *   d_x    = dg w1s[:Is] + du w1s[Is:]                       [T, H]
 *   d_w1s  = (dg | du)^T x,   d_w2s = d_out^T hs             [2*Is, H], [H, Is]
 * in dtype, rounded once from fp32 sums over operands in dtype (dg and du are
 * rounded to dtype).  Every element of an output is written (gradients are
 * not added to).  d_x may be NULL (not wanted: w1s may then be NULL too);
 * d_w1s and d_w2s may both be NULL (then x and hs may be NULL); not all three
 * where there are tokens.  Rows of padding: finite x with d_out of zero leaves
 * the weights' gradients untouched.  T == 0 writes zeros to d_w1s and d_w2s (NULL:
 * enqueues nothing).
 *   workspace: moe_shared_backward_workspace_size bytes, 256-byte aligned. */
moe_status moe_shared_ffn_backward(const moe_shape* shape, int32_t Is, double p,
                                   const uint64_t* rng, const void* x, const void* w1s,
                                   const void* w2s, const float* gu, const void* hs,
                                   const void* d_out, void* d_x, void* d_w1s, void* d_w2s,
                                   void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_SHARED_TRAIN_H */
