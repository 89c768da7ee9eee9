// The shared expert's backward pass (moe_shared_train.h): four matrix products
// in two launches.
//
//   dh = m s (d_out w2),  dg = dh u sigma(g) (1 + g (1 - sigma(g))),  du = dh SiLU(g)
//   d_x = [dg|du] w1,  d_w1 = [dg|du]^T x,  d_w2 = d_out^T h
//
// The weights are read as k-rows by the products that run back through them,
// x, h, d_out and dg|du by the weights' gradients: no transposed copies.  Each
// launch holds a product over the tokens' rows and a weight's gradient that
// does not wait for it (dg|du and d_w2, then d_x and d_w1), the longer sums
// first: the chip is left half idle twice and not four times, and the first
// product's epilogue, bound by memory (it reads g and u), runs beside the
// other's matrix work.  T = 2048, H = 4096, I = 768: 36 + 56 us, where d_gu alone
// and the three others took 24 + 76; T = 8192, I = 2048: 293 + 477 us (275 and 550
// GFLOP), 4 % longer than that way (159 + 580).  Sums over the tokens are not cut:
// a narrow layer with many tokens has few tiles of long sums (T = 8192, H = 256,
// I = 64: both launches 72 us in bf16, 221 us in fp32).
#include "shared_train.h"
#include "tile_gemm.h"

namespace moe {
namespace {

using tile::Operand;

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

// A product over rows of tokens (A k-contiguous, B k-rows), and a weight's
// gradient (both k-rows).
struct Part {
  Operand A, B;
  int K, mt, nt;
};

// Each die takes an eighth of either part's tiles, one part after the other.
template <class CX, class CW, class Epi>
__global__ __launch_bounds__(CX::NTHR, 1) void gradients_kernel(Part x, Part w, bool w_first, Epi epi_x,
                                                                tile::StoreOut<typename CX::E> epi_w) {
  static_assert(CX::LDS_BYTES == CW::LDS_BYTES && CX::NTHR == CW::NTHR && CX::BM == CW::BM && CX::BN == CW::BN, "one tile size");
  __shared__ __attribute__((aligned(1024))) char smem[CX::LDS_BYTES];
  const int die = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
  const int all_x = x.mt * x.nt, all_w = w.mt * w.nt, per_x = (all_x + kXcds - 1) / kXcds, per_w = (all_w + kXcds - 1) / kXcds;
  const bool is_w = w_first ? slot < per_w : slot >= per_x;
  int tm, tn;
  if (is_w) {
    const int s = w_first ? slot : slot - per_x, t = die * per_w + s;
    if (t >= all_w) return;
    tile::tile_of(t, w.mt, w.nt, tm, tn);
    tile::product<CW>(w.A, w.B, w.K, 0, tm * CW::BM, tn * CW::BN, epi_w, tile::NoExtra{}, smem);
  } else {
    const int s = w_first ? slot - per_w : slot, t = die * per_x + s;
    if (t >= all_x) return;
    tile::tile_of(t, x.mt, x.nt, tm, tn);
    tile::product<CX>(x.A, x.B, x.K, 0, tm * CX::BM, tn * CX::BN, epi_x, tile::NoExtra{}, smem);
  }
}

// has_x, has_w: which of the two are wanted.
template <class E, class Epi>
hipError_t run_both(Part x, bool has_x, const Epi& epi_x, Part w, bool has_w, const tile::StoreOut<E>& epi_w,
                    hipStream_t st) {
  const int size = tile::pair_tile<E>({has_x ? x.A.count : 0, x.B.count, x.K}, {has_w ? w.A.count : 0, w.B.count, w.K});
  return tile::with_tile<E>(size, [&](auto index) {
    typedef typename tile::TileCfg<E, decltype(index)::value, false, true>::type CX;
    typedef typename tile::TileCfg<E, decltype(index)::value, true, true>::type CW;
    unsigned slots = 0;
    auto split = [&](Part& p, bool has) {
      p.mt = has ? (p.A.count + CX::BM - 1) / CX::BM : 0;
      p.nt = (p.B.count + CX::BN - 1) / CX::BN;
      slots += (unsigned)(((long long)p.mt * p.nt + kXcds - 1) / kXcds);
    };
    split(x, has_x);
    split(w, has_w);
    if (slots == 0) return hipSuccess;
    hipLaunchKernelGGL((gradients_kernel<CX, CW, Epi>), dim3(slots * kXcds), dim3(CX::NTHR), 0, st, x, w, w.K > x.K,
                       epi_x, epi_w);
    return hipGetLastError();
  });
}

template <class E>
hipError_t backward(const Ffn& f, const Dropout& d, const void* x, const void* w1, const void* w2, const void* gu,
                    const void* hs, const void* d_out, void* d_gu, void* d_x, void* d_w1, void* d_w2, hipStream_t st) {
  const bool w = d_w1 != nullptr;
  const hipError_t e = run_both<E>(Part{Operand{d_out, f.H, f.T}, Operand{w2, f.I, f.I}, f.H, 0, 0}, true,
                                   SwigluBackward<E>{(const float*)gu, (E*)d_gu, f.I, d},
                                   Part{Operand{d_out, f.H, f.H}, Operand{hs, f.I, f.I}, f.T, 0, 0}, w,
                                   tile::StoreOut<E>{(E*)d_w2, nullptr, f.I}, st);
  if (e != hipSuccess) return e;
  return run_both<E>(Part{Operand{d_gu, 2 * f.I, f.T}, Operand{w1, f.H, f.H}, 2 * f.I, 0, 0}, d_x != nullptr,
                     tile::StoreOut<E>{(E*)d_x, nullptr, f.H},
                     Part{Operand{d_gu, 2 * f.I, 2 * f.I}, Operand{x, f.H, f.H}, f.T, 0, 0}, w,
                     tile::StoreOut<E>{(E*)d_w1, nullptr, f.H}, st);
}

}  // namespace

hipError_t launch_train_backward(const Ffn& f, const Dropout& d, const void* x, const void* w1, const void* w2,
                                 const void* gu, const void* hs, const void* d_out, void* d_gu, void* d_x, void* d_w1,
                                 void* d_w2, hipStream_t st) {
  return f.bf16 ? backward<uint16_t>(f, d, x, w1, w2, gu, hs, d_out, d_gu, d_x, d_w1, d_w2, st)
                : backward<float>(f, d, x, w1, w2, gu, hs, d_out, d_gu, d_x, d_w1, d_w2, st);
}

}  // namespace moe
