// 4-bit expert weights with group scales: storage arithmetic, operand
// conversion and the internal launchers (storage and semantics: moe_q4.h).
#pragma once

#include "lds_barrier.h"
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

// 16 bytes a lane of a code tile.
template <bool NONTEMPORAL>
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  if constexpr (NONTEMPORAL) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
  } else {
    return *reinterpret_cast<const uint4*>(p);
  }
}

// Element i of an operand as the fp32 value of its code (exact).
template <int FMT>
__device__ __forceinline__ float q4_value(const bf16x8& b, int i) {
  const float v = (float)b[i];
  return FMT == kQ4Int ? v - 136.0f : v;
}

// Keeps the additions that produce v in this block.  (The compiler may sink
// them past a branch, right behind the matrix instruction whose result they
// read, and then leaves out the wait states that this instruction needs.)
__device__ __forceinline__ void pin(f32x4& v) { asm volatile("" : "+v"(v)); }

// Sum of v over the 4, 8 or 16 neighbouring lanes that hold one group (DPP: no
// LDS round trip; mirrors do after the first two steps, whose sums are equal
// in a quad).
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  v = dpp_add<0xb1>(v);                           // quad_perm [1, 0, 3, 2]
  v = dpp_add<0x4e>(v);                           // quad_perm [2, 3, 0, 1]
  if constexpr (LANES >= 8) v = dpp_add<0x141>(v);   // row_half_mirror
  if constexpr (LANES >= 16) v = dpp_add<0x140>(v);  // row_mirror
  return v;
}

// -136 times the sum of 8 bf16 values, then over the lanes of one group (16 / GPB
// chunks of 8): what the accumulator of an INT4 group starts at.
template <int GPB>
__device__ __forceinline__ float q4_group_start(const uint4& v) {
  const bf16x2 c = __builtin_bit_cast(bf16x2, 0xc308c308u);  // -136, twice
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w[j]), c, s, false);
  asm volatile("" : "+v"(s));  // the reader below stays in this block (the wait states that the product needs)
  return lanes_sum<16 / GPB>(s);
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
