// Dropout with the residual added, and its backward pass (moe_shared_train.h).
//
// out[e] = residual[e] + (u[e] >= cut ? y[e] * scale : 0), u[e] the element's
// 16 random bits (philox.h).  The backward pass is the same kernel on d_out
// without a residual: the mask is computed again, nothing is stored.  Bound by
// HBM: T = 4096, H = 4096 bf16 takes 17.6 us with a residual (101 MB, 5.7 TB/s) and
// 12.8 us without (67 MB, 5.2 TB/s); eight elements a Philox block keep the
// generator below that.
#include "shared_train.h"
#include "tile_gemm.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kVecs = 4;

// A thread's kVecs vectors of eight elements lie kThreads vectors apart, so
// that every access of a wave is contiguous.
template <class E, bool RES>
__global__ __launch_bounds__(kThreads) void dropout_kernel(Dropout d, long long vecs, const E* y, const E* residual,
                                                           E* out) {
  const DropKey key = d.rng ? drop_key(d) : DropKey{};
  const long long v0 = (long long)blockIdx.x * (kThreads * kVecs) + threadIdx.x;
  tile::Vec8<E> a[kVecs], r[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const long long v = v0 + i * kThreads;
    if (v < vecs) {
      a[i].load(y + v * 8);
      if (RES) r[i].load(residual + v * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const long long v = v0 + i * kThreads;
    if (v < vecs) {
      uint4 b = make_uint4(0, 0, 0, 0);  // no dropout: cut is 0
      if (d.rng) b = philox((uint64_t)v, key);
      f32x4 o[2];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = dropped(a[i][e], b, e, d);
        o[e >> 2][e & 3] = RES ? r[i][e] + t : t;
      }
      tile::store8(out + v * 8, o[0], o[1]);
    }
  }
}

template <class E>
void run(const Dropout& d, long long n, const void* y, const void* residual, void* out, hipStream_t st) {
  const long long vecs = n / 8;
  const unsigned grid = (unsigned)((vecs + kThreads * kVecs - 1) / (kThreads * kVecs));
  if (residual)
    hipLaunchKernelGGL((dropout_kernel<E, true>), dim3(grid), dim3(kThreads), 0, st, d, vecs, (const E*)y,
                       (const E*)residual, (E*)out);
  else
    hipLaunchKernelGGL((dropout_kernel<E, false>), dim3(grid), dim3(kThreads), 0, st, d, vecs, (const E*)y,
                       (const E*)nullptr, (E*)out);
}

}  // namespace

hipError_t launch_dropout(bool bf16, const Dropout& d, long long n, const void* y, const void* residual, void* out,
                          hipStream_t st) {
  if (bf16)
    run<uint16_t>(d, n, y, residual, out, st);
  else
    run<float>(d, n, y, residual, out, st);
  return hipGetLastError();
}

}  // namespace moe
