// 4-bit expert weights with group scales: storage arithmetic, operand
// conversion and the internal launchers (storage and semantics: moe_q4.h).
#pragma once

#include "moe_common.h"

namespace moe {

constexpr int kQ4Int = 0, kQ4E2m1 = 1;
constexpr int kQ4TileK = 128;       // columns of a 1 KB code tile (16 rows)
constexpr int kQ4TileBytes = 1024;

struct Q4 {
  int format, group;
  int kb(int K) const { return (K + kQ4TileK - 1) / kQ4TileK; }             // code tiles along K
  int stride(int K) const { return (kb(K) + 3) / 4 * 4 * (kQ4TileK / group); }  // scales per row
};

// One 32-bit word of codes as 8 bf16 operands.  INT4 yields 128 + code: the
// four bits dropped into the mantissa of bf16 128 (one ulp is 1 there), two
// codes per and-or; the 136 too much is taken off per group by the caller.
// E2M1 converts on the gfx950 instruction, two codes at a time.
struct Q4Consts {
  // the and-or instruction takes one scalar and no literal: the mask is kept
  // in a scalar register, the exponent bits in a vector register (as literals
  // they cost an and and an or)
  uint32_t mask, base;
  __device__ __forceinline__ Q4Consts() {
    asm("s_mov_b32 %0, 0xf000f" : "=s"(mask));
    asm("v_mov_b32 %0, 0x43004300" : "=v"(base));
  }
};
template <int FMT>
__device__ __forceinline__ bf16x8 q4_operand(uint32_t w, const Q4Consts& k) {
  uint4 r;
  if constexpr (FMT == kQ4Int) {
    r.x = (w & k.mask) | k.base;
    r.y = ((w >> 4) & k.mask) | k.base;
    r.z = ((w >> 8) & k.mask) | k.base;
    r.w = ((w >> 12) & k.mask) | k.base;
  } else {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3));
  }
  return __builtin_bit_cast(bf16x8, r);
}

// Element i of an operand as the fp32 value of its code (exact).
template <int FMT>
__device__ __forceinline__ float q4_value(const bf16x8& b, int i) {
  const float v = (float)b[i];
  return FMT == kQ4Int ? v - 136.0f : v;
}

// The GPB scales of one row's code tile, as fp32.
template <int GPB>
__device__ __forceinline__ void q4_load_scales(const uint16_t* p, float (&s)[GPB]) {
  if constexpr (GPB == 1) {
    s[0] = bf16_bits_to_float(*p);
  } else if constexpr (GPB == 2) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    s[0] = __uint_as_float(v << 16);
    s[1] = __uint_as_float(v & 0xffff0000u);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    s[0] = __uint_as_float(v.x << 16);
    s[1] = __uint_as_float(v.x & 0xffff0000u);
    s[2] = __uint_as_float(v.y << 16);
    s[3] = __uint_as_float(v.y & 0xffff0000u);
  }
}
template <int GPB>
__device__ __forceinline__ void q4_load_scales(const float* p, float (&s)[GPB]) {
#pragma unroll
  for (int i = 0; i < GPB; ++i) s[i] = p[i];
}

// Grouped products over any number of rows per expert (q4_w13.hip, q4_down.hip).
hipError_t launch_q4_w13(const Shape& s, const Q4& q, const void* x, const int32_t* perm, const int32_t* offsets,
                         const void* codes, const void* scales, void* h, hipStream_t st);
hipError_t launch_q4_down(const Shape& s, const Q4& q, const void* h, const int32_t* offsets, const void* codes,
                          const void* scales, void* y, hipStream_t st);

// Small-token path of the whole layer (q4_decode.hip).
bool q4_decode_supported(const Shape& s);
hipError_t launch_q4_decode(const Shape& s, const Q4& q, const void* x, const float* wg, const float* bias,
                            const void* w1c, const void* w1s, const void* w2c, const void* w2s, void* out,
                            float* logits, int32_t* ids, float* w, int32_t* counts, int32_t* offsets, int32_t* perm,
                            int32_t* inv, void* h, void* scratch, hipStream_t st);

// Quantisation of a stack of matrices [N, K] (q4_quantize.hip); gate_up: w1's row order.
hipError_t launch_q4_quantize(const Q4& q, bool bf16, const void* w, long long matrices, int N, int K, bool gate_up,
                              void* codes, void* scales, hipStream_t st);

}  // namespace moe
