/*
 * moe_lora.h -- low-rank adapters of many requests at once beside the shared
 * expert's two projections, C ABI.
 *
 * The shared expert's weights (moe_shared.h) are the ones every token passes
 * through; a request may bring its own low-rank change of them.  Every token
 * names its adapter, and one call serves them all:
 *   z[t] = W x[t] + scale[a] * B[a] (A[a] x[t]),   a = adapter_ids[t]
 * A token whose id is outside [0, adapters) has none: z[t] = W x[t].
 *
 * Conventions are those of moe_mi355x.h: device pointers to caller-owned,
 * 16-byte aligned, contiguous row-major memory; `stream` is a hipStream_t
 * passed as void*; host-side validation first, and on any error nothing is
 * enqueued and no output is touched; T == 0 is valid and enqueues nothing.  Of
 * `shape`, T, H and dtype matter here (all fields are checked).  An output
 * overlaps no input, except where it says so.  The same call gives the same
 * bits, and what a token gets depends on its own adapter's values alone (others'
 * may be NaN), not on the other tokens of a batch of as many.  A workspace belongs to one call at a
 * time: calls that may overlap (other streams, other captured graphs) need
 * their own.
 *
 * Adapters: A [adapters, rank, K] and B [adapters, N, rank] in dtype, K and N
 * the projection's input and output widths; scale [adapters] fp32 (alpha /
 * rank); adapter_ids [T] int32.  One A serves gate and up; separate ones
 * are stacked (rank 2r, B with a block of zeros beside each).  Adapters of
 * lower rank are padded with zeros.  Sums are in fp32; in a bf16 layer of
 * more than 32 tokens scale * A x enters the second product as the sum of two
 * bf16 values (its rounding, at most bf16's largest number, and the rounding of
 * the rest, 2^-16 off; where scale * A x is infinite the rest is, and B times
 * it is what it is in fp32).
 *
 * Envelope, beside moe_mi355x.h's and moe_shared_train.h's for Is: rank a
 * multiple of 8 up to 128, up to 1024 adapters, T * max(H, Is) elements below
 * 4 GiB; otherwise MOE_ERR_UNSUPPORTED.  Non-positive numbers are
 * MOE_ERR_INVALID_ARG.
 */
#ifndef MOE_LORA_H
#define MOE_LORA_H

#include "moe_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_LORA_MAX_ADAPTERS 1024
#define MOE_LORA_MAX_RANK 128

typedef struct {
  int32_t adapters; /* adapters that A, B and scale hold */
  int32_t rank;
} moe_lora_spec;

/* Workspace bytes of the calls below (never fewer for more tokens), or 0 if an argument is invalid or
 * unsupported.  Pure host function. */
size_t moe_lora_workspace_size(const moe_shape* shape, int32_t Is, const moe_lora_spec* spec);

/* Gate and up projection with adapters, and SwiGLU:
 *   hs[t, i] = SiLU(z[t, i]) * z[t, Is + i]
 * x [T, H], w1s [2*Is, H], a1 [adapters, rank, H], b1 [adapters, 2*Is, rank];
 * output hs [T, Is] dtype, rounded once.
 *   workspace: moe_lora_workspace_size bytes, 256-byte aligned. */
moe_status moe_lora_w13_swiglu(const moe_shape* shape, int32_t Is, const moe_lora_spec* spec,
                               const void* x, const void* w1s, const void* a1, const void* b1,
                               const float* scale, const int32_t* adapter_ids, void* hs,
                               void* workspace, size_t workspace_bytes, void* stream);

/* Down projection with adapters:  out[t] = z[t] + residual[t]
 * hs [T, Is], w2s [H, Is], a2 [adapters, rank, Is], b2 [adapters, H, rank];
 * residual [T, H] dtype or NULL; output out [T, H] dtype, rounded once; out may
 * be residual. */
moe_status moe_lora_down(const moe_shape* shape, int32_t Is, const moe_lora_spec* spec,
                         const void* hs, const void* w2s, const void* a2, const void* b2,
                         const float* scale, const int32_t* adapter_ids, const void* residual,
                         void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Both in a row, the same adapters for both projections: hs as
 * moe_lora_w13_swiglu writes it, out as moe_lora_down does from it.  With the
 * output of moe_forward as residual, out is the layer with its shared expert. */
moe_status moe_shared_ffn_lora(const moe_shape* shape, int32_t Is, const moe_lora_spec* spec,
                               const void* x, const void* w1s, const void* w2s, const void* a1,
                               const void* b1, const void* a2, const void* b2, const float* scale,
                               const int32_t* adapter_ids, const void* residual, void* hs,
                               void* out, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LORA_H */
