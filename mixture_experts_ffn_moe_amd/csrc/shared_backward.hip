// The shared expert's backward pass (moe_shared_train.h): four matrix products
// in two launches.
//
//   dh = m s (d_out w2),  dg = dh u sigma(g) (1 + g (1 - sigma(g))),  du = dh SiLU(g)
//   d_x = [dg|du] w1,  d_w1 = [dg|du]^T x,  d_w2 = d_out^T h
//
// The weights are read as k-rows by the products that run back through them,
// x, h, d_out and dg|du by the weights' gradients: no transposed copies.  The
// three products of the second line do not depend on each other; they share a
// launch, whose tiles of the longest sums go first, so that the chip is left
// half idle once and not three times.
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

template <class E>
hipError_t dgu(const Ffn& f, const Dropout& d, const void* d_out, const void* w2, const void* gu, void* d_gu,
               hipStream_t st) {
  return tile::run_product<E, false, true>(Operand{d_out, f.H, f.T}, Operand{w2, f.I, f.I}, f.H, 0,
                                           SwigluBackward<E>{(const float*)gu, (E*)d_gu, f.I, d}, st);
}

struct Part {
  Operand A, B;
  int K, mt, nt;
  void* out;
};
struct Parts {
  Part p[3];
  int dx;  // which of them is d_x (its A is k-contiguous; -1: none of them)
};

// Each die takes an eighth of every part, parts in order.
template <class CX, class CW>
__global__ __launch_bounds__(CX::NTHR, 1) void gradients_kernel(Parts parts) {
  typedef typename CX::E E;
  static_assert(CX::LDS_BYTES == CW::LDS_BYTES && CX::NTHR == CW::NTHR && CX::BM == CW::BM && CX::BN == CW::BN, "one tile size");
  __shared__ __attribute__((aligned(1024))) char smem[CX::LDS_BYTES];
  int slot = blockIdx.x / kXcds;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const Part& p = parts.p[i];
    const int all = p.mt * p.nt, per = (all + kXcds - 1) / kXcds;
    if (slot < per) {
      const int t = (blockIdx.x % kXcds) * per + slot;
      if (t >= all) return;
      int tm, tn;
      tile::tile_of(t, p.mt, p.nt, tm, tn);
      const tile::StoreOut<E> epi{(E*)p.out, nullptr, p.B.count};
      if (i == parts.dx)
        tile::product<CX>(p.A, p.B, p.K, 0, tm * CX::BM, tn * CX::BN, epi, tile::NoExtra{}, smem);
      else
        tile::product<CW>(p.A, p.B, p.K, 0, tm * CW::BM, tn * CW::BN, epi, tile::NoExtra{}, smem);
      return;
    }
    slot -= per;
  }
}

template <class E>
hipError_t gradients(const Ffn& f, const void* x, const void* w1, const void* hs, const void* d_out, const void* d_gu,
                     void* d_x, void* d_w1, void* d_w2, hipStream_t st) {
  Part dx{Operand{d_gu, 2 * f.I, f.T}, Operand{w1, f.H, f.H}, 2 * f.I, 0, 0, d_x};
  Part a{Operand{d_gu, 2 * f.I, 2 * f.I}, Operand{x, f.H, f.H}, f.T, 0, 0, d_w1};
  Part b{Operand{d_out, f.H, f.H}, Operand{hs, f.I, f.I}, f.T, 0, 0, d_w2};
  Parts q = dx.K > f.T ? Parts{{dx, a, b}, 0} : Parts{{a, b, dx}, 2};
  const int size = tile::cheapest<E>([&](const tile::TileCost& c) {
    // the tiles' time spread over the chip, and half a tile of the longest sum for the last round
    long long sum = 0, longest = 0;
    for (const Part& p : q.p) {
      if (p.out == nullptr) continue;
      const long long tiles = (long long)((p.A.count + c.bm - 1) / c.bm) * ((p.B.count + c.bn - 1) / c.bn);
      const long long steps = ((long long)p.K * sizeof(E) + 127) / 128;
      sum += tiles * tile::tile_ns(c, steps, c.resident) / c.resident;
      const long long one = tile::tile_ns(c, steps, 1);
      longest = longest > one ? longest : one;
    }
    const long long spread = sum / tile::kCus;
    return spread > longest / 2 ? spread + longest / 2 : longest;
  });
  return tile::with_tile<E>(size, [&](auto index) {
    typedef typename tile::TileCfg<E, decltype(index)::value, false, true>::type CX;
    typedef typename tile::TileCfg<E, decltype(index)::value, true, true>::type CW;
    unsigned slots = 0;
    for (Part& p : q.p) {
      if (p.out == nullptr) continue;
      p.mt = (p.A.count + CX::BM - 1) / CX::BM;
      p.nt = (p.B.count + CX::BN - 1) / CX::BN;
      slots += (unsigned)(((long long)p.mt * p.nt + kXcds - 1) / kXcds);
    }
    hipLaunchKernelGGL((gradients_kernel<CX, CW>), dim3(slots * kXcds), dim3(CX::NTHR), 0, st, q);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_train_dgu(const Ffn& f, const Dropout& d, const void* d_out, const void* w2, const void* gu,
                            void* d_gu, hipStream_t st) {
  return f.bf16 ? dgu<uint16_t>(f, d, d_out, w2, gu, d_gu, st) : dgu<float>(f, d, d_out, w2, gu, d_gu, st);
}
hipError_t launch_train_gradients(const Ffn& f, const void* x, const void* w1, const void* hs, const void* d_out,
                                  const void* d_gu, void* d_x, void* d_w1, void* d_w2, hipStream_t st) {
  return f.bf16 ? gradients<uint16_t>(f, x, w1, hs, d_out, d_gu, d_x, d_w1, d_w2, st)
                : gradients<float>(f, x, w1, hs, d_out, d_gu, d_x, d_w1, d_w2, st);
}

}  // namespace moe
