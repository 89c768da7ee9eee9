// The shared expert as a gated feed-forward block that is trained
// (moe_shared_train.h): six matrix products with their pointwise parts fused.
//
//   forward   z = x w1^T = (g | u),  h = m s SiLU(g) u,  out = h w2^T + residual
//   backward  dh = m s (d_out w2),  dg = dh u sigma(g) (1 + g (1 - sigma(g))),
//             du = dh SiLU(g),  d_x = [dg|du] w1,  d_w1 = [dg|du]^T x,  d_w2 = d_out^T h
//
// g and u are kept in fp32: rounded to bf16 they raised the error of d_x and
// d_w1 from 2.4e-3 (dg, du and the result rounded once each) to 3.0e-3; their
// write and read are 2.5 % of the step at T = 8192, H = 4096, I = 2048.
#include "shared_train.h"
#include "tile_gemm.h"

namespace moe {
namespace {

using tile::Cfg;
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
struct SwigluBackward {
  static constexpr bool PAIR = false;
  const float* gu;
  E* d_gu;
  int I;
  Dropout d;
  struct Pre {
    tile::Vec8<float> g, u;
  };
  __device__ __forceinline__ Pre load(int row, int col) const {
    const float* p = gu + (size_t)row * (2 * (size_t)I) + col;
    Pre r;
    r.g.load(p);
    r.u.load(p + I);
    return r;
  }
  __device__ __forceinline__ void store(int row, int col, f32x4* v, const Pre& p) const {
    if (d.rng) {
      const uint4 b = philox(((size_t)row * I + col) >> 3, drop_key(d));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = dropped(v[i >> 2][i & 3], b, i, d);
    }
    f32x4 dg[2], du[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = p.g[i], dh = v[i >> 2][i & 3];
      const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
      dg[i >> 2][i & 3] = dh * p.u[i] * (s * (1.0f + g * (1.0f - s)));
      du[i >> 2][i & 3] = dh * (g * s);
    }
    E* q = d_gu + (size_t)row * (2 * (size_t)I) + col;
    tile::store8(q, dg[0], dg[1]);
    tile::store8(q + I, du[0], du[1]);
  }
};

// Tile sizes by the number of tiles: the largest that still gives most of
// the 256 CUs one.
template <bool TA, bool TB, class Epi>
hipError_t run(const Operand& A, const Operand& B, int K, int half, const Epi& epi, uint16_t, hipStream_t st) {
  const long long M = A.count, N = Epi::PAIR ? 2ll * half : B.count;
  auto tiles = [&](int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  if (tiles(256, 256) >= 192) return tile::launch_product<Cfg<uint16_t, 256, 256, 2, 4, 32, 64, 4, TA, TB>>(A, B, K, half, epi, st);
  if (tiles(128, 128) >= 192) return tile::launch_product<Cfg<uint16_t, 128, 128, 2, 2, 32, 128, 4, TA, TB>>(A, B, K, half, epi, st);
  return tile::launch_product<Cfg<uint16_t, 64, 64, 2, 2, 16, 128, 4, TA, TB>>(A, B, K, half, epi, st);
}
template <bool TA, bool TB, class Epi>
hipError_t run(const Operand& A, const Operand& B, int K, int half, const Epi& epi, float, hipStream_t st) {
  const long long M = A.count, N = Epi::PAIR ? 2ll * half : B.count;
  auto tiles = [&](int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  if (tiles(128, 128) >= 192) return tile::launch_product<Cfg<float, 128, 128, 2, 2, 16, 128, 4, TA, TB>>(A, B, K, half, epi, st);
  return tile::launch_product<Cfg<float, 64, 64, 2, 2, 16, 128, 4, TA, TB>>(A, B, K, half, epi, st);
}

template <class E>
hipError_t w13(const Ffn& f, const Dropout& d, const void* x, const void* w1, void* gu, void* hs, hipStream_t st) {
  return run<false, false>(Operand{x, f.H, f.T}, Operand{w1, f.H, 2 * f.I}, f.H, f.I,
                           TrainSwiglu<E>{(float*)gu, (E*)hs, f.I, d}, E{}, st);
}
template <class E>
hipError_t down(const Ffn& f, const void* hs, const void* w2, const void* residual, void* out, hipStream_t st) {
  return run<false, false>(Operand{hs, f.I, f.T}, Operand{w2, f.I, f.H}, f.I, 0,
                           tile::StoreOut<E>{(E*)out, (const E*)residual, f.H}, E{}, st);
}
template <class E>
hipError_t dgu(const Ffn& f, const Dropout& d, const void* d_out, const void* w2, const void* gu, void* d_gu,
               hipStream_t st) {
  return run<false, true>(Operand{d_out, f.H, f.T}, Operand{w2, f.I, f.I}, f.H, 0,
                          SwigluBackward<E>{(const float*)gu, (E*)d_gu, f.I, d}, E{}, st);
}
template <class E>
hipError_t dx(const Ffn& f, const void* d_gu, const void* w1, void* d_x, hipStream_t st) {
  return run<false, true>(Operand{d_gu, 2 * f.I, f.T}, Operand{w1, f.H, f.H}, 2 * f.I, 0,
                          tile::StoreOut<E>{(E*)d_x, nullptr, f.H}, E{}, st);
}
template <class E>
hipError_t dw(const Ffn& f, const void* x, const void* hs, const void* d_out, const void* d_gu, void* d_w1,
              void* d_w2, hipStream_t st) {
  hipError_t e = run<true, true>(Operand{d_out, f.H, f.H}, Operand{hs, f.I, f.I}, f.T, 0,
                                 tile::StoreOut<E>{(E*)d_w2, nullptr, f.I}, E{}, st);
  if (e != hipSuccess) return e;
  return run<true, true>(Operand{d_gu, 2 * f.I, 2 * f.I}, Operand{x, f.H, f.H}, f.T, 0,
                         tile::StoreOut<E>{(E*)d_w1, nullptr, f.H}, E{}, st);
}

}  // namespace

#define BY_TYPE(call, ...) (f.bf16 ? call<uint16_t>(__VA_ARGS__) : call<float>(__VA_ARGS__))

hipError_t launch_train_w13(const Ffn& f, const Dropout& d, const void* x, const void* w1, void* gu, void* hs,
                            hipStream_t st) {
  return BY_TYPE(w13, f, d, x, w1, gu, hs, st);
}
hipError_t launch_train_down(const Ffn& f, const void* hs, const void* w2, const void* residual, void* out,
                             hipStream_t st) {
  return BY_TYPE(down, f, hs, w2, residual, out, st);
}
hipError_t launch_train_dgu(const Ffn& f, const Dropout& d, const void* d_out, const void* w2, const void* gu,
                            void* d_gu, hipStream_t st) {
  return BY_TYPE(dgu, f, d, d_out, w2, gu, d_gu, st);
}
hipError_t launch_train_dx(const Ffn& f, const void* d_gu, const void* w1, void* d_x, hipStream_t st) {
  return BY_TYPE(dx, f, d_gu, w1, d_x, st);
}
hipError_t launch_train_dw(const Ffn& f, const void* x, const void* hs, const void* d_out, const void* d_gu,
                           void* d_w1, void* d_w2, hipStream_t st) {
  return BY_TYPE(dw, f, x, hs, d_out, d_gu, d_w1, d_w2, st);
}

}  // namespace moe
