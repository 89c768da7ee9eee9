// Quantisation of dense weights into the 4-bit storage of moe_q4.h.
//
// One wave per 1 KB code tile (16 rows x 128 columns), lane l holding the
// columns 32 j + 8 (l / 16) + i of row l % 16 that it will store: a group's
// magnitude is then a maximum over some of a lane's values and the row's four
// lanes.  The nearest code is found from the fp64 quotient, which is exact
// enough to tell a tie from its neighbours for any fp32 weight and scale.
// Runs once per weight: w1 of 64 experts, 1536 x 4096 in bf16 (805 MB), takes 0.90 -
// 0.95 ms (1.1 TB/s; 0.21 at a copy's rate).  Nothing forces the division, which is
// most of its instructions: products of the scale with the midpoints would be exact
// as well.
#include "q4.h"

namespace moe {
namespace {

template <typename XT>
__device__ __forceinline__ XT round_scale(float s);
template <>
__device__ __forceinline__ float round_scale<float>(float s) { return s; }
template <>
__device__ __forceinline__ uint16_t round_scale<uint16_t>(float s) { return float_to_bf16_bits(s); }

template <int FMT>
__device__ __forceinline__ uint32_t encode(float w, float s) {
  if (!(s > 0.0f)) return FMT == kQ4Int ? 8u : 0u;
  const double q = (double)w / (double)s;
  if constexpr (FMT == kQ4Int) {
    const double r = rint(q);
    return (uint32_t)(8 + (int)(r < -7.0 ? -7.0 : r > 7.0 ? 7.0 : r));
  } else {
    // the seven midpoints between neighbouring magnitudes; a tie goes to the even code
    const double a = fabs(q);
    const uint32_t c = (uint32_t)(a > 0.25) + (uint32_t)(a >= 0.75) + (uint32_t)(a > 1.25) + (uint32_t)(a >= 1.75) +
                       (uint32_t)(a > 2.5) + (uint32_t)(a >= 3.5) + (uint32_t)(a > 5.0);
    return c != 0 && q < 0.0 ? c | 8u : c;
  }
}

template <typename XT, int FMT, int GPB>
__global__ __launch_bounds__(256) void q4_quantize(const XT* __restrict__ w, long long tiles, int N, int K, int KB,
                                                   int S, int gate_up, uint8_t* __restrict__ codes,
                                                   XT* __restrict__ scales) {
  const long long tile = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);  // (matrix, row tile, column tile)
  if (tile >= tiles) return;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int kb = (int)(tile % KB);
  const long long rt = tile / KB;           // row tile over all matrices
  const int per = N / 16, it = (int)(rt % per);
  const long long mat = rt / per;
  const int row = gate_up ? (r < 8 ? 8 * it + r : N / 2 + 8 * it + r - 8) : 16 * it + r;
  const XT* src = w + ((size_t)mat * N + row) * K;

  float v[4][8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = kb * kQ4TileK + 32 * j + 8 * g;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = k < K ? Elem<XT>::load(src + k + i) : 0.0f;  // K % 8 == 0
  }
  constexpr int JG = 4 / GPB;
  float s[GPB];
#pragma unroll
  for (int q = 0; q < GPB; ++q) {
    float m = 0.0f;
#pragma unroll
    for (int j = q * JG; j < (q + 1) * JG; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[j][i]));
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const XT st = round_scale<XT>(__fdiv_rn(m, FMT == kQ4Int ? 7.0f : 6.0f));
    s[q] = Elem<XT>::to_f(st);
    if (g == 0) scales[((size_t)rt * 16 + r) * S + kb * GPB + q] = st;
  }
  // the padding of the row's scales, written with its last tile
  if (kb == KB - 1 && g == 0)
    for (int p = KB * GPB; p < S; ++p) scales[((size_t)rt * 16 + r) * S + p] = (XT)0;
  uint32_t word[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    word[j] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int nib = FMT == kQ4Int ? (i >> 1) + 4 * (i & 1) : i;
      word[j] |= encode<FMT>(v[j][i], s[j / JG]) << (4 * nib);
    }
  }
  *reinterpret_cast<uint4*>(codes + (size_t)tile * kQ4TileBytes + lane * 16) =
      make_uint4(word[0], word[1], word[2], word[3]);
}

template <typename XT, int FMT>
hipError_t launch_fmt(const Q4& q, const void* w, long long matrices, int N, int K, bool gate_up, void* codes,
                      void* scales, hipStream_t st) {
  const int KB = q.kb(K), S = q.stride(K);
  const long long tiles = matrices * (N / 16) * KB;
  const dim3 grid((unsigned)((tiles + 3) / 4)), block(256);
#define Q4_GO(GPB)                                                                                                  \
  hipLaunchKernelGGL((q4_quantize<XT, FMT, GPB>), grid, block, 0, st, (const XT*)w, tiles, N, K, KB, S, (int)gate_up, \
                     (uint8_t*)codes, (XT*)scales)
  if (q.group == 128) Q4_GO(1);
  else if (q.group == 64) Q4_GO(2);
  else Q4_GO(4);
#undef Q4_GO
  return hipGetLastError();
}

}  // namespace

hipError_t launch_q4_quantize(const Q4& q, bool bf16, const void* w, long long matrices, int N, int K, bool gate_up,
                              void* codes, void* scales, hipStream_t st) {
  if (bf16)
    return q.format == kQ4Int ? launch_fmt<uint16_t, kQ4Int>(q, w, matrices, N, K, gate_up, codes, scales, st)
                              : launch_fmt<uint16_t, kQ4E2m1>(q, w, matrices, N, K, gate_up, codes, scales, st);
  return q.format == kQ4Int ? launch_fmt<float, kQ4Int>(q, w, matrices, N, K, gate_up, codes, scales, st)
                            : launch_fmt<float, kQ4E2m1>(q, w, matrices, N, K, gate_up, codes, scales, st);
}

}  // namespace moe
