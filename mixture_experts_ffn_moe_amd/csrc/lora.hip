// Low-rank adapters of many requests at once beside the shared expert's two
// projections (moe_lora.h).
//
//   z[t] = W x[t] + s_a B_a (A_a x[t]),  a = ids[t] (none where it is outside [0, L))
//
// More than kSmallTokens tokens (or fp32):
//   * plan: a counting sort of the tokens by adapter, tokens without one last
//     (perm, the sorted adapters, every adapter's first position);
//   * shrink: low-rank values v[position, :] = s_a A_a x, one workgroup for 32
//     tokens of one adapter and a part of K, fp32 partial sums;
//   * product: the tiled product of tile_gemm.h over the sorted tokens, whose
//     accumulators take B_a v before the epilogue.  A fragment of rows that
//     several adapters share computes each one's product and every row takes
//     its own: no other adapter's values, NaN or not, reach a row, and the
//     order of tokens within an adapter does not change any bit.
// Up to kSmallTokens tokens in bf16: no sort; shrink per token, then one
// kernel that streams W with the tokens as the matrix instruction's columns
// and adds B_a v in its epilogue.
#include "shared_train.h"
#include "tile_gemm.h"

namespace moe {
namespace {

using tile::Cfg;
using tile::Mma;
using tile::Operand;

constexpr int kSmallTokens = 16;
constexpr int kMaxParts = 8;

bool small_path(const Ffn& f) { return f.bf16 && f.T <= kSmallTokens; }

// Parts of K whose low-rank sums are kept apart, so that few tokens still
// spread over the chip: 256 workgroups, at least 256 columns a part.
int parts_of(const Ffn& f, int K) {
  const int units = small_path(f) ? f.T : (f.T + 31) / 32;
  int p = 256 / units;
  p = p < K / 256 ? p : K / 256;
  return p < 1 ? 1 : p > kMaxParts ? kMaxParts : p;
}

constexpr int kPlanThreads = 1024;
int plan_blocks(int T) {
  const int b = (T + 8191) / 8192;
  return b < 256 ? b : 256;
}

struct Space {
  int32_t *perm, *sorted, *first, *hist;
  float* v;
  size_t bytes;
};
Space space(const Ffn& f, const Lora& l, void* ws) {
  char* p = (char*)ws;
  size_t at = 0;
  auto take = [&](size_t n) {
    char* r = p + at;
    at = (at + n + 255) & ~(size_t)255;
    return r;
  };
  Space s;
  s.perm = (int32_t*)take((size_t)f.T * 4);
  s.sorted = (int32_t*)take((size_t)f.T * 4);
  s.first = (int32_t*)take((size_t)(l.L + 2) * 4);
  s.hist = (int32_t*)take((size_t)plan_blocks(f.T) * (l.L + 1) * 4);
  const int a = parts_of(f, f.H), b = parts_of(f, f.I);
  s.v = (float*)take((size_t)(a > b ? a : b) * f.T * l.r * 4);
  s.bytes = at;
  return s;
}

// ---------------------------------------------------------------------------
// Plan.

__device__ __forceinline__ int bin_of(int id, int L) { return id >= 0 && id < L ? id : L; }

// Adds one for every lane's bin and returns the lane's place before it: the
// lanes that share the first lane's bin (a request's tokens lie together)
// take one addition.
__device__ __forceinline__ int count_up(int* bins, int bin, bool on) {
  int place = 0;
  const uint64_t live = __ballot(on);
  if (live == 0) return 0;
  const int lead = __ffsll((long long)live) - 1;
  const int b0 = __shfl(bin, lead);
  const uint64_t same = __ballot(on && bin == b0);
  const int lane = threadIdx.x & 63;
  int base = 0;
  if (lane == lead) base = atomicAdd(&bins[b0], __popcll(same));
  base = __shfl(base, lead);
  if (on && bin == b0)
    place = base + __popcll(same & ((1ull << lane) - 1));
  else if (on)
    place = atomicAdd(&bins[bin], 1);
  return place;
}

__global__ __launch_bounds__(kPlanThreads) void plan_count(const int32_t* ids, int T, int L, int chunk, int32_t* hist) {
  __shared__ int bins[kLoraMaxAdapters + 1];
  for (int i = threadIdx.x; i <= L; i += kPlanThreads) bins[i] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * chunk, t1 = min(T, t0 + chunk);
  for (int t = t0 + threadIdx.x; t - (int)threadIdx.x < t1; t += kPlanThreads)
    count_up(bins, t < t1 ? bin_of(ids[t], L) : 0, t < t1);
  __syncthreads();
  for (int i = threadIdx.x; i <= L; i += kPlanThreads) hist[(size_t)blockIdx.x * (L + 1) + i] = bins[i];
}

// Every workgroup finds its first position in every bin from all counts, then
// places its chunk.  Block 0 writes the bins' first positions.
__global__ __launch_bounds__(kPlanThreads) void plan_place(const int32_t* ids, int T, int L, int chunk,
                                                           const int32_t* hist, int blocks, int32_t* perm,
                                                           int32_t* sorted, int32_t* first) {
  __shared__ int start[kLoraMaxAdapters + 1];
  __shared__ int wave_sum[kPlanThreads / 64];
  __shared__ int carry;
  if (threadIdx.x == 0) carry = 0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
  for (int i0 = 0; i0 <= L; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int total = 0, before = 0;
    if (i <= L)
      for (int b = 0; b < blocks; ++b) {
        const int n = hist[(size_t)b * (L + 1) + i];
        total += n;
        before += b < (int)blockIdx.x ? n : 0;
      }
    int incl = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int base = carry;
    for (int w = 0; w < wave; ++w) base += wave_sum[w];
    if (i <= L) {
      start[i] = base + incl - total + before;
      if (blockIdx.x == 0) first[i] = base + incl - total;
    }
    __syncthreads();
    if (threadIdx.x == kPlanThreads - 1) carry = base + incl;
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) first[L + 1] = T;
  const int t0 = blockIdx.x * chunk, t1 = min(T, t0 + chunk);
  for (int t = t0 + threadIdx.x; t - (int)threadIdx.x < t1; t += kPlanThreads) {
    const bool on = t < t1;
    const int bin = on ? bin_of(ids[t], L) : 0;
    const int at = count_up(start, bin, on);
    if (on) {
      perm[at] = t;
      sorted[at] = bin;
    }
  }
}

// ---------------------------------------------------------------------------
// Shrink: 32 tokens of one adapter, RB * 32 ranks, a part of K split over
// the waves.

constexpr int kShrinkWaves = 4;

template <class E, int RB>
__global__ __launch_bounds__(kShrinkWaves * 64) void shrink_kernel(const E* x, const E* a, const float* scale,
                                                                   const int32_t* perm, const int32_t* first, int T,
                                                                   int K, int L, int r, int parts, float* v) {
  constexpr int F = sizeof(E) == 2 ? 32 : 16, FT = 32 / F, FR = RB * 32 / F, EPC = 16 / sizeof(E);
  typedef Mma<E, F> M;
  constexpr int LD = RB * 32 + 4;
  __shared__ float sum[kShrinkWaves][32 * LD];
  __shared__ int found[3];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // unit -> (adapter, first position): the units of an adapter with n tokens
  // are ceil(n / 32), adapters in order; wave 0 walks 64 of them at a time
  if (wave == 0) {
    int u = blockIdx.x, got = 0, ad = 0, p0 = 0, p1 = 0;
    for (int i0 = 0; i0 < L && !got; i0 += 64) {
      const int i = i0 + lane;
      const int lo = i < L ? first[i] : 0, hi = i < L ? first[i + 1] : 0;
      int incl = (hi - lo + 31) / 32;
      const int mine = incl;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
      }
      const uint64_t hit = __ballot(incl > u);
      if (hit) {
        const int w = __ffsll((long long)hit) - 1;
        ad = i0 + w;
        const int off = (u - __shfl(incl - mine, w)) * 32;
        p0 = __shfl(lo, w) + off;
        p1 = min(p0 + 32, __shfl(hi, w));
        got = 1;
      } else {
        u -= __shfl(incl, 63);
      }
    }
    if (lane == 0) {
      found[0] = got ? ad : -1;
      found[1] = p0;
      found[2] = p1;
    }
  }
  __syncthreads();
  const int ad = found[0], p0 = found[1], p1 = found[2];
  if (ad < 0) return;
  const int steps = K / M::SUB, part = blockIdx.y;
  const int s0 = (int)((long long)steps * part / parts), s1 = (int)((long long)steps * (part + 1) / parts);
  const int k0 = s0 + (s1 - s0) * wave / kShrinkWaves, k1 = s0 + (s1 - s0) * (wave + 1) / kShrinkWaves;
  const E *px[FT], *pa[FR];
#pragma unroll
  for (int i = 0; i < FT; ++i)
    px[i] = x + (size_t)perm[min(p0 + F * i + lane % F, p1 - 1)] * K + (lane / F) * EPC;
#pragma unroll
  for (int j = 0; j < FR; ++j)
    pa[j] = a + ((size_t)ad * r + min(F * j + lane % F, r - 1)) * K + (lane / F) * EPC;
  typename M::acc acc[FT][FR];
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FR; ++j)
#pragma unroll
      for (int e = 0; e < F * F / 64; ++e) acc[i][j][e] = 0.0f;
#pragma unroll 4
  for (int s = k0; s < k1; ++s) {
    typename M::frag fx[FT], fa[FR];
#pragma unroll
    for (int i = 0; i < FT; ++i) fx[i] = *reinterpret_cast<const typename M::frag*>(px[i] + (size_t)s * M::SUB);
#pragma unroll
    for (int j = 0; j < FR; ++j) fa[j] = *reinterpret_cast<const typename M::frag*>(pa[j] + (size_t)s * M::SUB);
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
      for (int j = 0; j < FR; ++j) acc[i][j] = M::mul(fa[j], fx[i], acc[i][j]);
  }
  tile::settle();
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FR; ++j)
#pragma unroll
      for (int q = 0; q < F * F / 256; ++q) {
        const f32x4 t = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        *reinterpret_cast<f32x4*>(&sum[wave][(F * i + lane % F) * LD + F * j + 8 * q + 4 * (lane / F)]) = t;
      }
  __syncthreads();
  const float sc = scale[ad];
  for (int i = tid; i < 32 * (r / 4); i += kShrinkWaves * 64) {
    const int row = i / (r / 4), c = (i % (r / 4)) * 4;
    if (p0 + row >= p1) break;
    f32x4 t = *reinterpret_cast<const f32x4*>(&sum[0][row * LD + c]);
#pragma unroll
    for (int w = 1; w < kShrinkWaves; ++w) {
      const f32x4 o = *reinterpret_cast<const f32x4*>(&sum[w][row * LD + c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] += o[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] *= sc;
    *reinterpret_cast<f32x4*>(v + ((size_t)part * T + p0 + row) * r + c) = t;
  }
}

// ---------------------------------------------------------------------------
// The low-rank addition to a tile's accumulators.

template <class E>
struct AddLora {
  static constexpr bool ON = true;
  const int32_t *perm, *sorted;
  const float* v;  // [parts, T, r]
  const E* b;      // [L, rows, r]
  int T, L, r, rows, parts;

  __device__ __forceinline__ int a_row(int p) const { return perm[p]; }
  __device__ __forceinline__ int out_row(int p) const { return perm[p]; }

  // 16 bytes of low-rank values of position p from rank k (zeros past r),
  // rounded to the layer's type as the matrix operand they are.
  __device__ __forceinline__ typename Mma<E, 16>::frag values(int p, int k) const {
    constexpr int N = 16 / sizeof(E);
    typename Mma<E, 16>::frag f;
    float t[N] = {};
    if (k < r) {
      for (int s = 0; s < parts; ++s) {
        const float* q = v + ((size_t)s * T + p) * r + k;
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          const f32x4 o = *reinterpret_cast<const f32x4*>(q + e);
#pragma unroll
          for (int i = 0; i < 4; ++i) t[e + i] += o[i];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if constexpr (sizeof(E) == 2) f[e] = (__bf16)t[e];
      else f[e] = t[e];
    }
    return f;
  }

  // m: the wave's first position; brow(j): this lane's row of b in fragment j.
  template <class C, class Row>
  __device__ __forceinline__ void add(typename C::M::acc (&acc)[C::FM][C::FN], int m, Row brow, int lane) const {
    constexpr int EPC = C::EPC;
    const int kl = (lane / C::F) * EPC;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const int p = min(m + C::F * i + lane % C::F, T - 1);
      const int mine = sorted[p];
      int cur = __builtin_amdgcn_readfirstlane(mine);
      while (cur < L) {
        typename C::M::acc d[C::FN];
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int e = 0; e < C::F * C::F / 64; ++e) d[j][e] = 0.0f;
        for (int k = 0; k < r; k += C::M::SUB) {
          const typename C::M::frag fv = values(p, k + kl);
#pragma unroll
          for (int j = 0; j < C::FN; ++j) {
            typename C::M::frag fb = {};
            if (k + kl < r)
              fb = *reinterpret_cast<const typename C::M::frag*>(b + ((size_t)cur * rows + brow(j)) * r + k + kl);
            d[j] = C::M::mul(fb, fv, d[j]);
          }
        }
        tile::settle();
        // every lane holds one row: it takes the product of its own adapter
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int e = 0; e < C::F * C::F / 64; ++e) acc[i][j][e] = mine == cur ? acc[i][j][e] + d[j][e] : acc[i][j][e];
        const uint64_t later = __ballot(mine > cur);
        if (later == 0) break;
        cur = __builtin_amdgcn_readlane(mine, __ffsll((long long)later) - 1);
      }
    }
  }
};

template <class E>
struct SwigluOut {
  static constexpr bool PAIR = true;
  E* hs;
  int I;
  struct Pre {};
  __device__ __forceinline__ Pre load(int, int) const { return Pre{}; }
  __device__ __forceinline__ void store(int row, int col, f32x4* v, const Pre&) const {
    f32x4 h[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i >> 2][i & 3] = silu_f32(v[i >> 2][i & 3]) * v[2 + (i >> 2)][i & 3];
    tile::store8(hs + (size_t)row * I + col, h[0], h[1]);
  }
};

template <class E, class Epi>
hipError_t big(const Ffn& f, const Lora& l, const void* x, int K, const void* w, int rows, const void* a,
               const void* b, const float* scale, const Epi& epi, void* ws, hipStream_t st) {
  const Space s = space(f, l, ws);
  const int parts = parts_of(f, K);
  const int units = (f.T + 31) / 32 + (l.L < f.T ? l.L : f.T);
  const dim3 grid(units, parts), blk(kShrinkWaves * 64);
#define SHRINK(RB)                                                                                                 \
  hipLaunchKernelGGL((shrink_kernel<E, RB>), grid, blk, 0, st, (const E*)x, (const E*)a, scale, s.perm, s.first, \
                     f.T, K, l.L, l.r, parts, s.v)
  if (l.r <= 32) SHRINK(1);
  else if (l.r <= 64) SHRINK(2);
  else SHRINK(4);
#undef SHRINK
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const AddLora<E> add{s.perm, s.sorted, s.v, (const E*)b, f.T, l.L, l.r, rows, parts};
  const Operand A{x, K, f.T}, B{w, K, rows};
  const int half = Epi::PAIR ? rows / 2 : 0;
  auto tiles = [&](int bm, int bn) { return (long long)((f.T + bm - 1) / bm) * ((rows + bn - 1) / bn); };
  if constexpr (sizeof(E) == 2) {
    if (tiles(256, 256) >= 192) return tile::launch_product<Cfg<E, 256, 256, 2, 4, 32, 64, 4, false, false>>(A, B, K, half, epi, st, add);
    if (tiles(128, 128) >= 192) return tile::launch_product<Cfg<E, 128, 128, 2, 2, 32, 128, 4, false, false>>(A, B, K, half, epi, st, add);
  } else {
    if (tiles(128, 128) >= 192) return tile::launch_product<Cfg<E, 128, 128, 2, 2, 16, 128, 4, false, false>>(A, B, K, half, epi, st, add);
  }
  return tile::launch_product<Cfg<E, 64, 64, 2, 2, 16, 128, 4, false, false>>(A, B, K, half, epi, st, add);
}

// ---------------------------------------------------------------------------
// Up to kSmallTokens tokens.

// v[part, t, j] = s_a A_a[j] . x[t] over a part of K: one workgroup a (token,
// part), a wave the ranks wave, wave + 4, ...
__global__ __launch_bounds__(256) void shrink_small(const uint16_t* x, const uint16_t* a, const float* scale,
                                                    const int32_t* ids, int T, int K, int L, int r, int parts,
                                                    float* v) {
  const int t = blockIdx.x, part = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ad = ids[t];
  if (ad < 0 || ad >= L) return;
  const int chunks = K / 8;
  const int c0 = (int)((long long)chunks * part / parts), c1 = (int)((long long)chunks * (part + 1) / parts);
  const float sc = scale[ad];
  for (int j = wave; j < r; j += 4) {
    float s = 0.0f;
    for (int c = c0 + lane; c < c1; c += 64) {
      tile::Vec8<uint16_t> p, q;
      p.load(x + (size_t)t * K + c * 8);
      q.load(a + ((size_t)ad * r + j) * K + c * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(p[e], q[e], s);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    if (lane == 0) v[((size_t)part * T + t) * r + j] = s * sc;
  }
}

// 16 rows of W (PAIR: 8 gate rows and their up rows), all tokens: the waves
// split K, their sums meet in LDS, and a thread finishes one (token, column).
template <bool PAIR>
__global__ __launch_bounds__(1024) void stream_kernel(const uint16_t* x, const uint16_t* w, const uint16_t* b,
                                                      const int32_t* ids, const float* v, const uint16_t* residual,
                                                      uint16_t* out, int T, int K, int N, int L, int r, int parts) {
  extern __shared__ float smem[];  // [waves][16][20] sums, then [16][r] low-rank values
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const int half = N / 2;
  const int n0 = blockIdx.x * (PAIR ? 8 : 16);
  auto wrow = [&](int i) { return PAIR ? (i < 8 ? n0 + i : half + n0 + i - 8) : n0 + i; };
  const uint16_t* pw = w + (size_t)wrow(lane & 15) * K + (lane >> 4) * 8;
  const uint16_t* px = x + (size_t)min(lane & 15, T - 1) * K + (lane >> 4) * 8;
  const int steps = K / 32;
  const int k0 = steps * wave / nw, k1 = steps * (wave + 1) / nw;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = k0; s < k1; ++s) {
    const bf16x8 fw = *reinterpret_cast<const bf16x8*>(pw + (size_t)s * 32);
    const bf16x8 fx = *reinterpret_cast<const bf16x8*>(px + (size_t)s * 32);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw, fx, acc, 0, 0, 0);
  }
  tile::settle();
  // lane: token lane % 16, rows 4 * (lane / 16) + e
  *reinterpret_cast<f32x4*>(smem + (wave * 16 + (lane & 15)) * 20 + 4 * (lane >> 4)) = acc;
  float* low = smem + nw * 16 * 20;
  for (int i = tid; i < T * r; i += blockDim.x) {
    const int ad = ids[i / r];
    float s = 0.0f;
    if (ad >= 0 && ad < L)
      for (int p = 0; p < parts; ++p) s += v[(size_t)p * T * r + i];
    low[i] = s;
  }
  __syncthreads();
  if (tid >= 256) return;
  const int t = tid >> 4, i = tid & 15;  // token, row of the sixteen
  float s = 0.0f;
  if (t < T) {
    for (int q = 0; q < nw; ++q) s += smem[(q * 16 + t) * 20 + i];
    const int ad = ids[t];
    if (ad >= 0 && ad < L) {
      const uint16_t* pb = b + ((size_t)ad * N + wrow(i)) * r;
      float d = 0.0f;
      for (int k = 0; k < r; k += 8) {
        tile::Vec8<uint16_t> q;
        q.load(pb + k);
#pragma unroll
        for (int e = 0; e < 8; ++e) d = fmaf(q[e], low[t * r + k + e], d);
      }
      s += d;
    }
  }
  if (PAIR) {
    const float up = __shfl_xor(s, 8);
    if (t < T && i < 8) out[(size_t)t * half + n0 + i] = float_to_bf16_bits(silu_f32(s) * up);
  } else if (t < T) {
    if (residual) s += bf16_bits_to_float(residual[(size_t)t * N + n0 + i]);
    out[(size_t)t * N + n0 + i] = float_to_bf16_bits(s);
  }
}

template <bool PAIR>
hipError_t small(const Ffn& f, const Lora& l, const void* x, int K, const void* w, int rows, const void* a,
                 const void* b, const float* scale, const int32_t* ids, const void* residual, void* out, void* ws,
                 hipStream_t st) {
  const Space s = space(f, l, ws);
  const int parts = parts_of(f, K);
  hipLaunchKernelGGL(shrink_small, dim3(f.T, parts), dim3(256), 0, st, (const uint16_t*)x, (const uint16_t*)a, scale,
                     ids, f.T, K, l.L, l.r, parts, s.v);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int steps = K / 32, nw = steps >= 64 ? 16 : steps >= 16 ? 8 : 4;
  const int lds = (nw * 16 * 20 + f.T * l.r) * 4;
  hipLaunchKernelGGL((stream_kernel<PAIR>), dim3(rows / 16), dim3(nw * 64), lds, st, (const uint16_t*)x,
                     (const uint16_t*)w, (const uint16_t*)b, ids, s.v, (const uint16_t*)residual, (uint16_t*)out,
                     f.T, K, rows, l.L, l.r, parts);
  return hipGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(const Ffn& f, const Lora& l) { return space(f, l, nullptr).bytes; }

hipError_t launch_lora_plan(const Ffn& f, const Lora& l, const int32_t* ids, void* ws, hipStream_t st) {
  if (small_path(f)) return hipSuccess;
  const Space s = space(f, l, ws);
  const int blocks = plan_blocks(f.T), chunk = (f.T + blocks - 1) / blocks;
  hipLaunchKernelGGL(plan_count, dim3(blocks), dim3(kPlanThreads), 0, st, ids, f.T, l.L, chunk, s.hist);
  hipLaunchKernelGGL(plan_place, dim3(blocks), dim3(kPlanThreads), 0, st, ids, f.T, l.L, chunk, s.hist, blocks,
                     s.perm, s.sorted, s.first);
  return hipGetLastError();
}

hipError_t launch_lora_w13(const Ffn& f, const Lora& l, const void* x, const void* w1, const void* a, const void* b,
                           const float* scale, const int32_t* ids, void* hs, void* ws, hipStream_t st) {
  if (small_path(f)) return small<true>(f, l, x, f.H, w1, 2 * f.I, a, b, scale, ids, nullptr, hs, ws, st);
  if (f.bf16) return big<uint16_t>(f, l, x, f.H, w1, 2 * f.I, a, b, scale, SwigluOut<uint16_t>{(uint16_t*)hs, f.I}, ws, st);
  return big<float>(f, l, x, f.H, w1, 2 * f.I, a, b, scale, SwigluOut<float>{(float*)hs, f.I}, ws, st);
}

hipError_t launch_lora_down(const Ffn& f, const Lora& l, const void* hs, const void* w2, const void* a, const void* b,
                            const float* scale, const int32_t* ids, const void* residual, void* out, void* ws,
                            hipStream_t st) {
  if (small_path(f)) return small<false>(f, l, hs, f.I, w2, f.H, a, b, scale, ids, residual, out, ws, st);
  if (f.bf16)
    return big<uint16_t>(f, l, hs, f.I, w2, f.H, a, b, scale,
                         tile::StoreOut<uint16_t>{(uint16_t*)out, (const uint16_t*)residual, f.H}, ws, st);
  return big<float>(f, l, hs, f.I, w2, f.H, a, b, scale,
                    tile::StoreOut<float>{(float*)out, (const float*)residual, f.H}, ws, st);
}

}  // namespace moe
