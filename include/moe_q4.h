/*
 * moe_q4.h -- the routed layer over 4-bit expert weights with group scales,
 * C ABI.
 *
 * In the AR-decode regime the layer's time is the time its active experts'
 * weights take to arrive from HBM; held in 4 bits they are a quarter of
 * bf16.  Everything else of the layer is unchanged: router, permutation,
 * SwiGLU, finalize, the types of x, h, y and out.
 *
 * A weight is  w[n, k] = scale[n, k / group] * value(code[n, k])  with
 *   MOE_Q4_INT4:  value(c) = c - 8, c in [0, 16)
 *   MOE_Q4_E2M1:  bit 3 the sign, bits 2..0 one of 0, 0.5, 1, 1.5, 2, 3, 4, 6
 * and scales in the layer's dtype, one per `group` (32, 64 or 128) columns.
 * Products: the codes' values are exact operands; each group's sum is taken in
 * fp32, multiplied by its scale and added in fp32, so a weight is never
 * rounded beyond its 4 bits.
 *
 * Storage.  A weight stack is a list of matrices [N, K], N % 16 == 0, in the
 * order of the dense layer's: w1 [mu, E] of N = 2*Im, K = H; w2 [mu, E] of
 * N = H, K = Im.  With KB = ceil(K / 128):
 *  - codes: [matrix][N/16 row tiles][KB][1024 bytes].  A 1 KB tile is 16 rows
 *    x 128 columns as the 64 lanes of a wave load it: lane l owns bytes
 *    [16 l, 16 l + 16), four little-endian 32-bit words j = 0..3, word j
 *    holding the 8 codes of row l % 16, columns 128 kb + 32 j + 8 (l / 16) + i,
 *    i = 0..7.  Nibble (4 bits, nibble 0 the lowest) of element i:
 *    INT4 (i >> 1) + 4 (i & 1), E2M1 i.  Columns >= K hold the code of zero
 *    (INT4 8, E2M1 0).
 *  - rows: w2's tiles take 16 rows in order; a tile of w1 holds 8 gate rows
 *    8 q .. 8 q + 7 and then their 8 up rows Im + 8 q .. Im + 8 q + 7.
 *  - scales: [matrix][N][S], rows in the order of the tiles, S =
 *    4 * ceil(KB / 4) * (128 / group); entries past K / group are zero.
 * moe_q4_quantize_w13 and moe_q4_quantize_down write this storage from dense
 * weights.
 *
 * Conventions are those of moe_mi355x.h: device pointers to caller-owned,
 * 16-byte aligned, contiguous memory; `stream` is a hipStream_t passed as
 * void*; host-side validation first, and on any error nothing is enqueued and
 * no output is touched; T == 0 is valid and enqueues nothing (the quantisers
 * quantise whatever T is).
 *
 * Envelope, beside moe_mi355x.h's: group divides H and Im; otherwise
 * MOE_ERR_UNSUPPORTED.  An unknown format or a group that is not 32, 64 or
 * 128 is MOE_ERR_INVALID_ARG.  x and h must be finite and below 2^100 in
 * magnitude (the INT4 codes enter the matrix pipe as 128 + code, and 136 times
 * the operand's sum is taken off again in fp32).
 *
 * Any number of tokens runs; the kernels are built for few rows per expert
 * (blocks of up to 48 rows, 32 in fp32, share one read of the codes), where the
 * weights' bytes count.  Long prompts are faster in bf16: the whole layer at
 * H = 4096, E = 64, k = 8, Im = 768, INT4 groups of 128 against moe_forward, us:
 *   T = 8 59 / 151, 64 101 / 319, 256 140 / 335, 1024 347 / 381,
 *   2048 639 / 468, 4096 1146 / 723;
 * with two micro-shards 1024 555 / 604, 2048 1027 / 734.  A program that keeps
 * both weights changes over between 1024 and 2048 tokens.
 */
#ifndef MOE_Q4_H
#define MOE_Q4_H

#include "moe_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_Q4_INT4 = 0, MOE_Q4_E2M1 = 1 } moe_q4_format;

typedef struct {
  int32_t format; /* moe_q4_format */
  int32_t group;  /* columns per scale: 32, 64 or 128 */
} moe_q4_spec;

/* Bytes of the stored weights of one layer. */
typedef struct {
  size_t w1_codes, w1_scales, w2_codes, w2_scales;
} moe_q4_sizes;

/* Fills `sizes` for (shape, q4).  Pure host function. */
moe_status moe_q4_get_sizes(const moe_shape* shape, const moe_q4_spec* q4, moe_q4_sizes* sizes);

/* Quantises dense weights of the layer's dtype into the storage above,
 * group by group: M the group's largest magnitude, scale = M / 7 (INT4) or
 * M / 6 (E2M1) rounded to dtype, and the code whose value times that scale is
 * nearest to the weight (ties to the even code magnitude; INT4 uses -7..7).
 * A group whose scale rounds to zero stores zero codes.  Weights are finite.
 *   w1 [mu, E, 2*Im, H], w2 [mu, E, H, Im]. */
moe_status moe_q4_quantize_w13(const moe_shape* shape, const moe_q4_spec* q4, const void* w1,
                               void* codes, void* scales, void* stream);
moe_status moe_q4_quantize_down(const moe_shape* shape, const moe_q4_spec* q4, const void* w2,
                                void* codes, void* scales, void* stream);

/* moe_grouped_gemm_w13_swiglu over 4-bit weights: same x, perm, offsets and h. */
moe_status moe_q4_w13_swiglu(const moe_shape* shape, const moe_q4_spec* q4, const void* x,
                             const int32_t* perm, const int32_t* offsets, const void* w1_codes,
                             const void* w1_scales, void* h, void* stream);

/* moe_grouped_gemm_down over 4-bit weights: same h, offsets and y (so that
 * moe_finalize and moe_finalize_backward read it). */
moe_status moe_q4_down(const moe_shape* shape, const moe_q4_spec* q4, const void* h,
                       const int32_t* offsets, const void* w2_codes, const void* w2_scales, void* y,
                       void* stream);

/* moe_forward over 4-bit weights, in a workspace of moe_workspace_size(shape)
 * bytes with the same layout.  The small-token regime (bf16, T <= 16,
 * H % 2048 == 0, T rounded up to 4 times H and T times mu times Im rounded up
 * to 128 both <= 65536) takes a path of its own, as in moe_forward: routing is
 * the same bits as the step-wise path, the output matches it within rounding
 * (sums in another order, y never stored).  Up to 1024 tokens of other bf16
 * batches the router's fp64 sums run in another order than moe_route's: a logit
 * can differ by its last fp32 bit only where its sum lies within the order's
 * difference (about 2^-40 of the terms' magnitudes) of a rounding border. */
moe_status moe_forward_q4(const moe_shape* shape, const moe_q4_spec* q4, const void* x,
                          const float* wg, const float* bias, const void* w1_codes,
                          const void* w1_scales, const void* w2_codes, const void* w2_scales,
                          void* out, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_Q4_H */
