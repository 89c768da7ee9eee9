// The shared expert as a gated feed-forward block that is trained
// (moe_shared_train.h), forward pass: two matrix products with their pointwise
// parts fused (the backward pass: shared_backward.hip).
//
//   z = x w1^T = (g | u),  h = m s SiLU(g) u,  out = h w2^T + residual
//
// g and u are kept in fp32: rounded to bf16 they raised the error of d_x and
// d_w1 from 2.4e-3 (dg, du and the result rounded once each) to 3.0e-3; their
// write and read are 2.5 % of the step at T = 8192, H = 4096, I = 2048.
#include "shared_train.h"
#include "tile_gemm.h"

namespace moe {
namespace {

// T = 8192, H = 4096, I = 2048, dropout: w13 268 us (275 GFLOP; the 168 MB that it
// writes leave with all tiles of a round at once), down with residual 156 us
// (137 GFLOP).

using tile::Operand;

template <class E>
struct TrainSwiglu {
  static constexpr bool PAIR = true;
  float* gu;
  E* hs;
  int I;
  Dropout d;
  struct Pre {};
  __device__ __forceinline__ Pre load(int, int) const { return Pre{}; }
  __device__ __forceinline__ void store(int row, int col, f32x4* v, const Pre&) const {
    float* p = gu + (size_t)row * (2 * (size_t)I) + col;
    tile::store8(p, v[0], v[1]);
    tile::store8(p + I, v[2], v[3]);
    f32x4 h[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i >> 2][i & 3] = silu_f32(v[i >> 2][i & 3]) * v[2 + (i >> 2)][i & 3];
    const size_t e = (size_t)row * I + col;
    if (d.rng) {
      const uint4 b = philox(e >> 3, drop_key(d));
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i >> 2][i & 3] = dropped(h[i >> 2][i & 3], b, i, d);
    }
    tile::store8(hs + e, h[0], h[1]);
  }
};

template <class E>
hipError_t w13(const Ffn& f, const Dropout& d, const void* x, const void* w1, void* gu, void* hs, hipStream_t st) {
  return tile::run_product<E, false, false>(Operand{x, f.H, f.T}, Operand{w1, f.H, 2 * f.I}, f.H, f.I,
                                            TrainSwiglu<E>{(float*)gu, (E*)hs, f.I, d}, st);
}
template <class E>
hipError_t down(const Ffn& f, const void* hs, const void* w2, const void* residual, void* out, hipStream_t st) {
  return tile::run_product<E, false, false>(Operand{hs, f.I, f.T}, Operand{w2, f.I, f.H}, f.I, 0,
                                            tile::StoreOut<E>{(E*)out, (const E*)residual, f.H}, st);
}

}  // namespace

hipError_t launch_train_w13(const Ffn& f, const Dropout& d, const void* x, const void* w1, void* gu, void* hs,
                            hipStream_t st) {
  return f.bf16 ? w13<uint16_t>(f, d, x, w1, gu, hs, st) : w13<float>(f, d, x, w1, gu, hs, st);
}
hipError_t launch_train_down(const Ffn& f, const void* hs, const void* w2, const void* residual, void* out,
                             hipStream_t st) {
  return f.bf16 ? down<uint16_t>(f, hs, w2, residual, out, st) : down<float>(f, hs, w2, residual, out, st);
}

}  // namespace moe
