// Low-rank adapters of many requests at once beside the shared expert's two
// projections (moe_lora.h).
//
//   z[t] = W x[t] + s_a B_a (A_a x[t]),  a = ids[t] (none where it is outside [0, L))
//
// More than kSmallTokens tokens (or fp32):
//   * plan: a counting sort of the tokens by adapter, tokens without one last
//     (perm, the sorted adapters, every adapter's first position);
//   * low-rank values v = s_a A_a x, fp32 partial sums over parts of K: by tiles of
//     32 sorted tokens of one adapter (after the plan, v by position), or, few of
//     them, by a wave for each (beside the plan in one launch, v by token);
//   * product: the tiled product of tile_gemm.h over the sorted tokens, whose
//     accumulators take B_a v before the epilogue.  A fragment of rows that
//     several adapters share computes each one's product and every row takes
//     its own: no other adapter's values, NaN or not, reach a row, and the
//     order of tokens within an adapter does not change any bit.
// Up to kSmallTokens tokens in bf16: no sort; a wave for each low-rank value,
// then one kernel that streams W with the tokens as the matrix instruction's
// columns and adds B_a v in its epilogue.
#include "shared_train.h"
#include "tile_gemm.h"

namespace moe {
namespace {

using tile::Cfg;
using tile::Mma;
using tile::Operand;

// Tokens up to which W is streamed.  32 tokens, H = 4096, Is = 768, both
// projections in a graph, this way and by tiles (24 workgroups for w13): rank 16 of 64
// adapters 19.0 and 34.3 us, rank 128 of 4 51.7 and 51.6.  64 tokens, 8 rows of W a
// workgroup: rank 16 of 64 31.5 and 35.9, but H = 2048, Is = 1536, rank 32 39.3 and 29.3.
constexpr int kSmallTokens = 32;
constexpr int kMaxParts = 8;

bool small_path(const Ffn& f) { return f.bf16 && f.T <= kSmallTokens; }

// Tokens of a workgroup of the sort (8192 tokens in one workgroup: 8.4 us; 300: 3.9 us).
constexpr int kPlanThreads = 1024, kPlanChunk = 8192;
int plan_blocks(int T) { return (T + kPlanChunk - 1) / kPlanChunk; }

// Few low-rank values of short adapters are computed by a wave each: every wave
// reads a row of A, from L2 mostly.  us of a call of w13 (N = 1536, bf16, in a graph)
// by waves and by tiles, on both sides of either border:
//   values (T r <= 8192): K = 4096, rank 16, 300 tokens 24.0 and 27.5, 512 29.6 and 33.6,
//     768 40.0 and 38.5; rank 8, 1024 tokens 36.0 and 38.2, 1500 52.6 and 57.5; K = 1024,
//     N = 512, rank 64, 100 tokens 16.0 and 17.9, 200 18.1 and 16.9;
//   elements of an adapter (r K <= 65536), there: K = 8192, rank 8, 300 tokens 38.3 and
//     40.7, 1024 61.6 and 56.6; 98304: K = 4096, rank 24, 128 tokens 25.8 and 27.8, 341 33.3
//     and 34.3; 131072: K = 4096, rank 32, 256 tokens 28.7 and 29.2, K = 8192, rank 16, 300
//     42.9 and 42.3, K = 16384, rank 8, 300 67.3 and 65.1, 1024 108 and 93; 262144: K = 4096,
//     rank 64, 64 tokens 40.8 and 39.3; 524288: rank 128, 40 tokens 42.7 and 34.5.
// fp32, K = 448, N = 320, rank 8, 77 tokens: 11.8 and 16.4; K = 4096, rank 16, 256 tokens: 56.5 and 60.7.
// The sort's launch with 300 tokens' values of rank 16 takes 7.8 to 8.3 us (in two: 4.8 and 5.3).
bool by_wave(const Ffn& f, const Lora& l, int K) {
  return small_path(f) || (f.T <= kPlanChunk && (long long)f.T * l.r <= 8192 && (long long)l.r * K <= 1 << 16);
}

// Parts of K whose low-rank sums are kept apart, so that few tokens still
// spread over the chip: 512 workgroups, at least 128 columns a part (512 by
// waves).
int parts_of(const Ffn& f, const Lora& l, int K) {
  const bool waves = by_wave(f, l, K);
  const int units = small_path(f) ? 1 : waves ? f.T : (f.T + 31) / 32, least = waves ? 512 : 128;
  int p = 512 / units;
  p = p < K / least ? p : K / least;
  return p < 1 ? 1 : p > kMaxParts ? kMaxParts : p;
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
  s.first = (int32_t*)take((size_t)(l.L + 1) * 4);
  s.hist = (int32_t*)take((size_t)plan_blocks(f.T) * (l.L + 1) * 4);
  // parts * T is at most this (512 workgroups of 32 tokens), which grows with T:
  // a workspace for many tokens serves fewer
  const size_t few = (size_t)f.T * kMaxParts;
  const size_t low = few < 512 * 32 ? few : 512 * 32;
  s.v = (float*)take((low > (size_t)f.T ? low : (size_t)f.T) * l.r * 4);
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

// Every workgroup counts its chunk, finds its first position in every bin from
// all chunks' counts (hist; a lone workgroup's are its own), and places its
// tokens.  Block 0 writes the bins' first positions.
__device__ __forceinline__ void place_tokens(const int32_t* ids, int T, int L, int chunk, const int32_t* hist,
                                             int blocks, int32_t* perm, int32_t* sorted, int32_t* first) {
  __shared__ int start[kLoraMaxAdapters + 1];
  __shared__ int wave_sum[kPlanThreads / 64];
  __shared__ int carry;
  constexpr int KEEP = kPlanChunk / kPlanThreads;  // a thread's tokens of a chunk
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t0 = blockIdx.x * chunk, t1 = min(T, t0 + chunk);
  int bin[KEEP], place[KEEP];
#pragma unroll
  for (int q = 0; q < KEEP; ++q) {
    const int t = t0 + q * kPlanThreads + threadIdx.x;
    bin[q] = t < t1 ? bin_of(ids[t], L) : -1;
  }
  for (int i = threadIdx.x; i <= L; i += kPlanThreads) start[i] = 0;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < KEEP; ++q) place[q] = count_up(start, bin[q], bin[q] >= 0);
  __syncthreads();
  for (int i0 = 0; i0 <= L; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int total = 0, before = 0;
    if (i <= L) {
      if (blocks == 1)
        total = start[i];
      else
        for (int b = 0; b < blocks; ++b) {
          const int n = hist[(size_t)b * (L + 1) + i];
          total += n;
          before += b < (int)blockIdx.x ? n : 0;
        }
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
#pragma unroll
  for (int q = 0; q < KEEP; ++q)
    if (bin[q] >= 0) {
      const int at = start[bin[q]] + place[q];
      perm[at] = t0 + q * kPlanThreads + threadIdx.x;
      sorted[at] = bin[q];
    }
}

__global__ __launch_bounds__(kPlanThreads) void plan_place(const int32_t* ids, int T, int L, int chunk,
                                                           const int32_t* hist, int blocks, int32_t* perm,
                                                           int32_t* sorted, int32_t* first) {
  place_tokens(ids, T, L, chunk, hist, blocks, perm, sorted, first);
}

// ---------------------------------------------------------------------------
// Low-rank values by waves.

// One row of A times x over the 8-column chunks c0 .. c1, by a wave.
template <class E>
__device__ __forceinline__ float low_rank_value(const E* x, const E* a, int c0, int c1, int lane) {
  float s = 0.0f;
#pragma unroll 4
  for (int c = c0 + lane; c < c1; c += 64) {
    tile::Vec8<E> p, q;
    p.load(x + c * 8);
    q.load(a + c * 8);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(p[e], q[e], s);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  return s;
}

// v[part, t, j] = s_a A_a[j] . x[t] over a part of K: workgroups (token, part,
// ranks by the number of waves).  PLAN: the first workgroup sorts the tokens
// instead.
template <class E, int WAVES, bool PLAN>
__global__ __launch_bounds__(WAVES * 64, 8) void low_kernel(const E* x, const E* a, const float* scale,
                                                         const int32_t* ids, int T, int K, int L, int r, int parts,
                                                         float* v, int32_t* perm, int32_t* sorted, int32_t* first) {
  static_assert(!PLAN || WAVES * 64 == kPlanThreads, "threads of the sort");
  int block = blockIdx.x;
  if constexpr (PLAN) {
    if (block == 0) {
      place_tokens(ids, T, L, T, nullptr, 1, perm, sorted, first);
      return;
    }
    --block;
  }
  const int t = block % T, part = block / T % parts, lane = threadIdx.x & 63;
  const int j = block / T / parts * WAVES + (threadIdx.x >> 6);
  const int ad = ids[t];
  if (ad < 0 || ad >= L || j >= r) return;
  const int chunks = K / 8;
  const int c0 = chunks * part / parts, c1 = chunks * (part + 1) / parts;
  const float s = low_rank_value(x + (size_t)t * K, a + ((size_t)ad * r + j) * K, c0, c1, lane);
  if (lane == 0) v[((size_t)part * T + t) * r + j] = s * scale[ad];
}

// ---------------------------------------------------------------------------
// Shrink: 32 tokens of one adapter, BN ranks, a part of K.  Operand fragments
// read straight from memory would touch 16 rows per 16 lanes (eight times the
// line accesses of whole rows: 27 us for 8192 tokens, K = 2048, rank 64), so the rows
// come through LDS like those of any tiled product.

struct Gather {
  static constexpr bool ON = false, MAPPED = true;
  const int32_t* perm;
  __device__ __forceinline__ int a_row(int p) const { return perm[p]; }
  __device__ __forceinline__ int out_row(int p) const { return p; }
  template <class C, class R0, class Row>
  __device__ __forceinline__ int begin(int, int, R0, Row, int, int) const { return 0; }
};
struct StoreLow {
  static constexpr bool PAIR = false;
  float* v;
  int r;
  float scale;
  struct Pre {};
  __device__ __forceinline__ Pre load(int, int) const { return Pre{}; }
  __device__ __forceinline__ void store(int row, int col, f32x4* s, const Pre&) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e >> 2][e & 3] *= scale;
    tile::store8(v + (size_t)row * r + col, s[0], s[1]);
  }
};

template <class C>
__global__ __launch_bounds__(C::NTHR) void shrink_kernel(const typename C::E* x, const typename C::E* a,
                                                         const float* scale, const int32_t* perm,
                                                         const int32_t* first, int T, int K, int L, int r, int parts,
                                                         float* v) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS_BYTES];
  // unit -> (adapter, first position): the units of an adapter with n tokens
  // are ceil(n / BM), adapters in order; every wave walks 64 of them at a time
  const int lane = threadIdx.x & 63;
  int u = blockIdx.x, ad = -1, p0 = 0, p1 = 0;
  for (int i0 = 0; i0 < L; i0 += 64) {
    const int i = i0 + lane;
    const int lo = i < L ? first[i] : 0, hi = i < L ? first[i + 1] : 0;
    const int mine = (hi - lo + C::BM - 1) / C::BM;
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    const uint64_t hit = __ballot(incl > u);
    if (hit) {
      const int w = __ffsll((long long)hit) - 1;
      ad = i0 + w;
      p0 = __shfl(lo, w) + (u - __shfl(incl - mine, w)) * C::BM;
      p1 = __shfl(hi, w);
      break;
    }
    u -= __shfl(incl, 63);
  }
  ad = __builtin_amdgcn_readfirstlane(ad);
  p0 = __builtin_amdgcn_readfirstlane(p0);
  p1 = min(__builtin_amdgcn_readfirstlane(p1), p0 + C::BM);
  if (ad < 0) return;
  const int part = blockIdx.y, tiles = (K + C::BK - 1) / C::BK;
  const int k0 = tiles * part / parts * C::BK, k1 = min(K, tiles * (part + 1) / parts * C::BK);
  const StoreLow epi{v + (size_t)part * T * r, r, scale[ad]};
  tile::product<C, StoreLow, Gather>(Operand{x + k0, K, p1}, Operand{a + (size_t)ad * r * K + k0, K, r}, k1 - k0, 0, p0,
                                     blockIdx.z * C::BN, epi, Gather{perm}, smem);
}

// ---------------------------------------------------------------------------
// The low-rank addition to a tile's accumulators.

// What the first of the two bf16 operands of a low-rank value t rounds.  Past
// bf16's largest number that number is taken: the rest t - 0x1.fep127 is then
// finite where t is, and infinite or NaN where t is (an infinite first operand
// would leave inf - inf).
__device__ __forceinline__ float first_part(float t) { return __builtin_amdgcn_fmed3f(t, -0x1.fep127f, 0x1.fep127f); }

template <class E>
struct AddLora {
  static constexpr bool ON = true, MAPPED = true;
  const int32_t *perm, *sorted, *first;
  const float* v;  // [parts, T, r], by position or by token
  const E* b;      // [L, rows, r]
  int T, L, r, rows, parts;
  bool by_token;

  __device__ __forceinline__ int a_row(int p) const { return perm[p]; }
  __device__ __forceinline__ int out_row(int p) const { return perm[p]; }

  // The runs of equal adapters among a tile's rows: run n is tile rows
  // start .. next start, start << 16 | adapter.
  template <int BM>
  struct Runs {
    uint32_t run[BM + 1];
    int count;
  };
  template <int BM>
  static __device__ __forceinline__ Runs<BM>& runs() {
    __shared__ Runs<BM> s;
    return s;
  }
  // Ranks of one substep in tiles of 16-row fragments: a wave reads the fragments
  // of B of its own rows' adapters straight from memory (16 short rows of B lie
  // together), the first ones ahead of the main loop, and needs neither LDS
  // nor barriers for them.  w13 of 300 tokens, K = 4096, rank 16, this way and
  // by the ring: 64 adapters 17.7 and 20.6 us, 300 adapters 18.7 and 28, one 17.1
  // and 17.1, none 17.4 and 15.6.
  template <class C>
  static __device__ __forceinline__ constexpr bool direct(int r) {
    return C::F == 16 && r <= C::M::SUB;
  }
  template <class C>
  struct Ahead {
    static constexpr int Q = C::FM < 4 ? 4 / C::FM : 1;  // adapters of a batch
    static constexpr int N = 16 / sizeof(E);
    int ad[C::FM], at[C::FM];   // of this lane's row: its adapter, its low-rank values
    uint32_t heads[C::FM];      // fragment rows where another adapter begins
    f32x4 low[C::FM][N / 4];    // the first part's values
    int id[C::FM][Q];           // the first adapters
    typename C::M::frag b[C::FM][Q][C::FN];
  };
  // The fragments of B of the next adapters among a fragment's rows.
  template <class C, class R0, class Row>
  __device__ __forceinline__ void take(uint32_t& heads, int ad, int (&id)[Ahead<C>::Q],
                                       typename C::M::frag (&f)[Ahead<C>::Q][C::FN], R0 b_r0, Row brow, int lane) const {
    const int k = Ahead<C>::N * (lane / 16);
#pragma unroll
    for (int q = 0; q < Ahead<C>::Q; ++q) {
      id[q] = -1;
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int e = 0; e < Ahead<C>::N; ++e) f[q][j][e] = 0.0f;
      if (heads == 0) continue;
      id[q] = __builtin_amdgcn_readlane(ad, __ffs((int)heads) - 1);
      heads &= heads - 1;
      const E* base = uniform_ptr(b + (size_t)id[q] * rows * r);
      if (k < r)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
          f[q][j] = *reinterpret_cast<const typename C::M::frag*>(base + (size_t)brow(b_r0(j) + lane % 16) * r + k);
    }
  }

  // Behind the first copies, ahead of the main loop.
  template <class C, class R0, class Row>
  __device__ __forceinline__ auto begin(int m0, int wave_m, R0 b_r0, Row brow, int wave, int lane) const {
    if constexpr (C::F == 16) {
      Ahead<C> h;
      if (!direct<C>(r)) {
        list_runs<C>(m0, wave, lane);
        return h;
      }
      const int k = Ahead<C>::N * (lane / 16);
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const int p = m0 + wave_m + 16 * i + lane % 16;
        h.ad[i] = p < T ? sorted[p] : L;
        h.at[i] = p < T && by_token ? perm[p] : p;
      }
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const int left = __shfl_up(h.ad[i], 1);
        h.heads[i] = (uint32_t)__ballot(h.ad[i] < L && (lane == 0 || h.ad[i] != left)) & 0xffffu;
        take<C>(h.heads[i], h.ad[i], h.id[i], h.b[i], b_r0, brow, lane);
#pragma unroll
        for (int c = 0; c < Ahead<C>::N / 4; ++c) {
          h.low[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};
          if (h.ad[i] < L && k < r) h.low[i][c] = reinterpret_cast<const f32x4*>(v + (size_t)h.at[i] * r + k)[c];
        }
      }
      return h;
    } else {
      list_runs<C>(m0, wave, lane);
      return 0;
    }
  }

  template <class C, class R0, class Row>
  __device__ __forceinline__ void add_direct(typename C::M::acc (&acc)[C::FM][C::FN], const Ahead<C>& h, R0 b_r0, Row brow,
                                             int lane) const {
    constexpr int N = Ahead<C>::N, Q = Ahead<C>::Q;
    const int k = N * (lane / 16);
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      if (h.id[i][0] < 0) continue;  // no adapter in these rows
      f32x4 t[N / 4];
#pragma unroll
      for (int c = 0; c < N / 4; ++c) t[c] = h.low[i][c];
      if (h.ad[i] < L && k < r)
        for (int s = 1; s < parts; ++s)
#pragma unroll
          for (int c = 0; c < N / 4; ++c)
            t[c] += reinterpret_cast<const f32x4*>(v + ((size_t)s * T + h.at[i]) * r + k)[c];
      typename C::M::frag value, rest;
#pragma unroll
      for (int e = 0; e < N; ++e) value[e] = sizeof(E) == 2 ? first_part(t[e / 4][e % 4]) : t[e / 4][e % 4];
      if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int e = 0; e < N; ++e) rest[e] = t[e / 4][e % 4] - (float)value[e];
      }
      uint32_t heads = h.heads[i];
      int id[Q];
      typename C::M::frag f[Q][C::FN];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        id[q] = h.id[i][q];
#pragma unroll
        for (int j = 0; j < C::FN; ++j) f[q][j] = h.b[i][q][j];
      }
      for (;;) {
        typename C::M::acc d[Q][C::FN];
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int j = 0; j < C::FN; ++j) {
            d[q][j] = typename C::M::acc{0.f, 0.f, 0.f, 0.f};
            if constexpr (sizeof(E) == 2) d[q][j] = C::M::mul(f[q][j], rest, d[q][j]);
            d[q][j] = C::M::mul(f[q][j], value, d[q][j]);
          }
        tile::settle();
        // every lane holds one row: it takes the product of its own adapter
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = h.ad[i] == id[q] ? acc[i][j][e] + d[q][j][e] : acc[i][j][e];
        if (heads == 0) break;
        take<C>(heads, h.ad[i], id, f, b_r0, brow, lane);
      }
    }
  }

  // Where not direct: the tile's runs, for add.
  template <class C>
  __device__ __forceinline__ void list_runs(int m0, int wave, int lane) const {
    if (wave != 0) return;
    Runs<C::BM>& s = runs<C::BM>();
    int n = 0;
#pragma unroll
    for (int r0 = 0; r0 < C::BM; r0 += 64) {
      const int row = r0 + lane, p = m0 + row;
      const int mine = row < C::BM && p < T ? sorted[p] : L;
      const int left = row > 0 && row < C::BM && p < T ? sorted[p - 1] : -1;
      const bool start = mine != left && mine < L;
      const uint64_t mask = __ballot(start);
      if (start) s.run[n + __popcll(mask & ((1ull << lane) - 1))] = (uint32_t)row << 16 | (uint32_t)mine;
      n += __popcll(mask);
    }
    // the end of the last run: tokens without an adapter come last
    const int end = min(first[L] - m0, C::BM);
    if (lane == 0) {
      s.run[n] = (uint32_t)(n ? end : 0) << 16;
      s.count = n;
    }
  }

  // Adds B_a v to the tile's accumulators; where not direct, with the ring's LDS in use for it: the
  // tile's low-rank values of RS ranks (summed over the parts), and a ring of
  // the B rows of the tile's adapters, copied ahead.  In bf16 a low-rank value is
  // the sum of two operands, its rounding and the rounding of what is left:
  // rounded once it raised the error of SwiGLU's output from 1.7e-3 (its own
  // rounding) to 3.1e-3 where the adapters' part is large.  b_r0(j): first tile row of this
  // wave's fragment j; brow(i): row of B of tile row i.
  template <class C, class H, class R0, class Row>
  __device__ __forceinline__ void add(typename C::M::acc (&acc)[C::FM][C::FN], const H& ahead, char* smem, int m0,
                                      int wave_m, R0 b_r0, Row brow, int wave, int lane) const {
    if constexpr (C::F == 16)
      if (direct<C>(r)) return add_direct<C>(acc, ahead, b_r0, brow, lane);
    typedef Cfg<E, C::BM, C::BN, C::WM, C::WN, C::F, 128, 2, false, false> S;  // tiles of 128-byte rows
    constexpr int RS = 128 / sizeof(E), V_BYTES = sizeof(E) == 2 ? 2 * S::A_BYTES : S::A_BYTES;
    constexpr int RING = (C::LDS_BYTES - V_BYTES) / S::B_BYTES < 6 ? (C::LDS_BYTES - V_BYTES) / S::B_BYTES : 6;
    static_assert(RING >= 2 && (RING - 2) * S::BQ < 64, "ring of B tiles");
    const Runs<C::BM>& list = runs<C::BM>();
    const int count = __builtin_amdgcn_readfirstlane(list.count);
    if (count == 0) return;
    const uint32_t lds = (uint32_t)(uintptr_t)smem + V_BYTES;
    for (int k0 = 0; k0 < r; k0 += RS) {
      const int left = min(RS, r - k0);
      if (k0) __syncthreads();
      uint32_t off[S::BQ];
      tile::copy_offsets<S, false, C::BN>(off, 0, 0, r, left, wave, lane, brow);
      int sent = 0;
      auto copy = [&]() {  // past the last run, its B again: every wait counts the same
        const uint32_t a = __builtin_amdgcn_readfirstlane(list.run[min(sent, count - 1)]) & 0xffffu;
        const char* p = uniform_ptr((const char*)(b + (size_t)a * rows * r + k0));
#pragma unroll
        for (int i = 0; i < S::BQ; ++i)
          dma16(lds + (uint32_t)((sent % RING) * S::B_BYTES) + (uint32_t)(wave + C::NW * i) * 1024u, p, off[i]);
        ++sent;
      };
      for (int n = 0; n < RING - 1; ++n) copy();
      // low-rank values, 16 bytes at a time, zeros past the rank
      constexpr int N = 16 / sizeof(E);
      for (int e = wave * 64 + lane; e < C::BM * 8; e += C::NTHR) {
        const int row = e >> 3, c = e & 7;
        f32x4 t[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        if (m0 + row < T && c * N < left) {
          const int at = by_token ? perm[m0 + row] : m0 + row;
          for (int s = 0; s < parts; ++s) {
            const float* q = v + ((size_t)s * T + at) * r + k0 + c * N;
#pragma unroll
            for (int h = 0; h < N / 4; ++h) t[h] += reinterpret_cast<const f32x4*>(q)[h];
          }
        }
        char* to = smem + row * 128 + (c ^ tile::swz_row<128>(row)) * 16;
        if constexpr (sizeof(E) == 2) {
          f32x4 near[2];
#pragma unroll
          for (int i = 0; i < 8; ++i) near[i >> 2][i & 3] = first_part(t[i >> 2][i & 3]);
          const uint2 a0 = pack_bf16x4(near[0]), a1 = pack_bf16x4(near[1]);
          tile::Vec8<uint16_t> a;
          a.d = make_uint4(a0.x, a0.y, a1.x, a1.y);
          *reinterpret_cast<uint4*>(to) = a.d;
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i >> 2][i & 3] -= a[i];
          const uint2 l0 = pack_bf16x4(t[0]), l1 = pack_bf16x4(t[1]);
          *reinterpret_cast<uint4*>(to + S::A_BYTES) = make_uint4(l0.x, l0.y, l1.x, l1.y);
        } else {
          *reinterpret_cast<f32x4*>(to) = t[0];
        }
      }
      for (int n = 0; n < count; ++n) {
        wait_vmcnt<(RING - 2) * S::BQ>();  // this run's B
        tile::slot_barrier();
        const int r0 = __builtin_amdgcn_readfirstlane(list.run[n]) >> 16, r1 = __builtin_amdgcn_readfirstlane(list.run[n + 1]) >> 16;
        copy();
        const char* tb = smem + V_BYTES + (n % RING) * S::B_BYTES;
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
          const int f0 = wave_m + C::F * i;
          if (f0 >= r1 || f0 + C::F <= r0) continue;
          typename C::M::acc d[C::FN];
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int e = 0; e < C::F * C::F / 64; ++e) d[j][e] = 0.0f;
          for (int ks = 0; ks * C::M::SUB < left; ++ks) {
            const int some = left - ks * C::M::SUB;
            const typename C::M::frag fv = tile::read_frag<S, false, C::BM>(smem, wave_m + C::F * i, ks, lane);
            typename C::M::frag rest;
            if constexpr (sizeof(E) == 2)
              rest = tile::read_frag<S, false, C::BM>(smem + S::A_BYTES, wave_m + C::F * i, ks, lane);
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
              typename C::M::frag fb = tile::read_frag<S, false, C::BN>(tb, b_r0(j), ks, lane);
              if (some < C::M::SUB) fb = tile::mask_k<S>(fb, some, lane);
              if constexpr (sizeof(E) == 2) d[j] = C::M::mul(fb, rest, d[j]);
              d[j] = C::M::mul(fb, fv, d[j]);
            }
          }
          tile::settle();
          // every lane holds one row: it takes the product of its own adapter
          const int row = f0 + lane % C::F;
          const bool mine = row >= r0 && row < r1;
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int e = 0; e < C::F * C::F / 64; ++e) acc[i][j][e] = mine ? acc[i][j][e] + d[j][e] : acc[i][j][e];
        }
      }
      wait_vmcnt<0>();
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

hipError_t sort_tokens(const Ffn& f, const Lora& l, const int32_t* ids, const Space& s, hipStream_t st) {
  const int blocks = plan_blocks(f.T), chunk = (f.T + blocks - 1) / blocks;
  if (blocks > 1) {
    hipLaunchKernelGGL(plan_count, dim3(blocks), dim3(kPlanThreads), 0, st, ids, f.T, l.L, chunk, s.hist);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(plan_place, dim3(blocks), dim3(kPlanThreads), 0, st, ids, f.T, l.L, chunk, s.hist, blocks,
                     s.perm, s.sorted, s.first);
  return hipGetLastError();
}

// plan: the tokens are not sorted yet.
template <class E, class Epi>
hipError_t big(const Ffn& f, const Lora& l, const void* x, int K, const void* w, int rows, const void* a,
               const void* b, const float* scale, const int32_t* ids, bool plan, const Epi& epi, void* ws,
               hipStream_t st) {
  const Space s = space(f, l, ws);
  const int parts = parts_of(f, l, K);
  const bool waves = by_wave(f, l, K);
  hipError_t e = hipSuccess;
  if (waves) {
    constexpr int W = kPlanThreads / 64;
    auto low = [&](auto kernel, int before) {
      hipLaunchKernelGGL(kernel, dim3(before + f.T * parts * ((l.r + W - 1) / W)), dim3(W * 64), 0, st, (const E*)x,
                         (const E*)a, scale, ids, f.T, K, l.L, l.r, parts, s.v, s.perm, s.sorted, s.first);
      return hipGetLastError();
    };
    e = plan ? low(low_kernel<E, W, true>, 1) : low(low_kernel<E, W, false>, 0);
  } else {
    if (plan) e = sort_tokens(f, l, ids, s, st);
    if (e != hipSuccess) return e;
    const int units = (f.T + 31) / 32 + (l.L < f.T ? l.L : f.T);
    auto shrink = [&](auto cfg) {
      typedef decltype(cfg) C;
      static_assert(C::BM == 32, "units of 32 tokens");
      hipLaunchKernelGGL(shrink_kernel<C>, dim3(units, parts, (l.r + C::BN - 1) / C::BN), dim3(C::NTHR), 0, st,
                         (const E*)x, (const E*)a, scale, s.perm, s.first, f.T, K, l.L, l.r, parts, s.v);
      return hipGetLastError();
    };
    e = l.r <= 32 ? shrink(Cfg<E, 32, 32, 1, 2, 16, 128, 4, false, false>{})
                  : shrink(Cfg<E, 32, 64, 1, 4, 16, 128, 4, false, false>{});
  }
  if (e != hipSuccess) return e;
  const AddLora<E> add{s.perm, s.sorted, s.first, s.v, (const E*)b, f.T, l.L, l.r, rows, parts, waves};
  const Operand A{x, K, f.T}, B{w, K, rows};
  const int half = Epi::PAIR ? rows / 2 : 0;
  return tile::run_product<E, false, false>(A, B, K, half, epi, st, add);
}

// ---------------------------------------------------------------------------
// Up to kSmallTokens tokens.

// ROWS rows of W (PAIR: half of them gate rows, then their up rows), all
// tokens: the waves split K in chunks of 64 columns, each with a ring of its
// own in LDS that direct copies fill with whole 128-byte rows (no workgroup
// barrier); their sums meet in LDS, and a thread finishes one (token, row).
// What the end needs (low-rank values, the first 32 ranks of B) is loaded right
// behind the first copies, so that the latencies overlap.  16 tokens, H = 4096,
// Is = 768, rank 32: 7.1 us for w13 (12.6 MB of weights, 2.7 us at the copy rate; 13 us
// with operands read straight from memory, 16 rows per 16 lanes) and 4.5 us down.
// Above 16 tokens x takes twice the LDS of a slot, and half as many waves have
// a ring each; a third slot in it changed nothing.
constexpr int kStreamRing = 2;
constexpr int stream_waves(int tokens) { return tokens == 16 ? 16 : 8; }

// TOK: the most tokens.  OWN: the low-rank values are computed here, by every
// workgroup for itself.
template <bool PAIR, int ROWS, int TOK, bool OWN>
__global__ __launch_bounds__(stream_waves(TOK) * 64) void stream_kernel(
    const uint16_t* x, const uint16_t* w, const uint16_t* a, const uint16_t* b, const float* scale, const int32_t* ids,
    const float* v, const uint16_t* residual, uint16_t* out, int T, int K, int N, int L, int r, int parts) {
  static_assert((ROWS == 8 || ROWS == 16) && (TOK == 16 || TOK == 32), "rows of W, tokens");
  constexpr int WAVES = stream_waves(TOK), FR = TOK / 16, XG = TOK / 8, WG = ROWS / 8;
  constexpr int SLOT = (ROWS + TOK) * 128, COPIES = WG + XG;
  constexpr int RING = WAVES * kStreamRing * SLOT;
  static_assert(TOK * ROWS <= WAVES * 64, "a thread for every result");
  __shared__ __attribute__((aligned(1024))) char ring[RING];
  __shared__ float low[TOK * kLoraMaxRank];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = N / 2, cols = PAIR ? ROWS / 2 : ROWS;
  const int n0 = blockIdx.x * cols;
  auto wrow = [&](int i) { return i < cols ? n0 + i : half + n0 + i - cols; };
  const int chunks = (K + 63) / 64;
  const uint32_t lds = (uint32_t)(uintptr_t)ring + (uint32_t)(wave * kStreamRing * SLOT);
  uint32_t woff[WG], xoff[XG];
  int col[XG];  // columns of this lane's 16 bytes, by row group
#pragma unroll
  for (int g = 0; g < XG; ++g) {
    const int row = g * 8 + (lane >> 3);
    col[g] = ((lane & 7) ^ tile::swz_row<128>(row)) * 8;
    if (g < WG) woff[g] = ((uint32_t)wrow(row) * (uint32_t)K + (uint32_t)col[g]) * 2u;
    xoff[g] = ((uint32_t)min(row, T - 1) * (uint32_t)K + (uint32_t)col[g]) * 2u;
  }
  // Copies of chunk c into slot c's place; the last chunk may hold 32 columns
  // only: what lies past them is read from the chunk's start and not used.
  auto copy = [&](int n) {
    const int c = wave + WAVES * n;
    const bool past = c * 64 + 64 > K;
    const uint32_t s = lds + (uint32_t)((n % kStreamRing) * SLOT);
    const char* pw = uniform_ptr((const char*)w + (size_t)c * 128);
    const char* px = uniform_ptr((const char*)x + (size_t)c * 128);
#pragma unroll
    for (int g = 0; g < WG; ++g) dma16(s + g * 1024u, pw, past && col[g] >= 32 ? woff[g] - col[g] * 2u : woff[g]);
#pragma unroll
    for (int g = 0; g < XG; ++g)
      dma16(s + ROWS * 128u + g * 1024u, px, past && col[g] >= 32 ? xoff[g] - col[g] * 2u : xoff[g]);
  };
  const int mine = wave < chunks ? (chunks - wave + WAVES - 1) / WAVES : 0;
#pragma unroll
  for (int n = 0; n < kStreamRing; ++n)
    if (n < mine) copy(n);

  const int t = tid / ROWS, i = tid % ROWS;  // token and row that this thread finishes
  const bool live = t < T;
  const int ad = live ? ids[t] : -1;
  const bool has = ad >= 0 && ad < L;
  const uint16_t* pb = b + ((size_t)(has ? ad : 0) * N + wrow(i)) * r;
  tile::Vec8<uint16_t> q[4];
  if (has) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c * 8 < r) q[c].load(pb + c * 8);
  }
  if constexpr (OWN) {
    for (int e = wave; e < T * r; e += WAVES) {
      const int to = e / r, id = ids[to];
      if (id >= 0 && id < L) {
        const float s = low_rank_value(x + (size_t)to * K, a + ((size_t)id * r + e % r) * K, 0, K / 8, lane) * scale[id];
        if (lane == 0) low[e] = s;
      }
    }
  } else {
    for (int e = tid; e < T * r; e += WAVES * 64) {
      const int id = ids[e / r];
      float s = 0.0f;
      if (id >= 0 && id < L)
        for (int p = 0; p < parts; ++p) s += v[(size_t)p * T * r + e];
      low[e] = s;
    }
  }

  f32x4 acc[FR];
#pragma unroll
  for (int f = 0; f < FR; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int fr = lane & 15;
  for (int n = 0; n < mine; ++n) {
    // chunk n has landed; behind it at most one chunk's copies are in flight
    if (n + 1 < mine && n > 0)
      wait_vmcnt<COPIES>();
    else
      wait_vmcnt<0>();
    __builtin_amdgcn_sched_barrier(0);
    const char* s = ring + wave * kStreamRing * SLOT + (n % kStreamRing) * SLOT;
    const int steps = min(2, (K - (wave + WAVES * n) * 64) / 32);
    for (int ks = 0; ks < steps; ++ks) {
      const int wr = fr % ROWS, cw = ((ks * 4 + (lane >> 4)) ^ tile::swz_row<128>(wr)) * 16;
      const bf16x8 fw = *reinterpret_cast<const bf16x8*>(s + wr * 128 + cw);
#pragma unroll
      for (int f = 0; f < FR; ++f) {
        const int xr = f * 16 + fr, cx = ((ks * 4 + (lane >> 4)) ^ tile::swz_row<128>(xr)) * 16;
        const bf16x8 fx = *reinterpret_cast<const bf16x8*>(s + ROWS * 128 + xr * 128 + cx);
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw, fx, acc[f], 0, 0, 0);
      }
    }
    if (n + kStreamRing < mine) {
      __builtin_amdgcn_s_waitcnt(0xF | (7 << 4) | (0 << 8) | (3 << 14));  // the slot's reads are done
      __builtin_amdgcn_sched_barrier(0);
      copy(n + kStreamRing);
    }
  }
  tile::settle();
  __syncthreads();  // every wave is past its ring
  // lane: token lane % 16, rows 4 * (lane / 16) + e
  float* sums = reinterpret_cast<float*>(ring);
  static_assert(WAVES * TOK * 20 * 4 <= RING, "sums in the ring's place");
#pragma unroll
  for (int f = 0; f < FR; ++f)
    *reinterpret_cast<f32x4*>(sums + (wave * TOK + f * 16 + fr) * 20 + 4 * (lane >> 4)) = acc[f];
  __syncthreads();
  if (tid >= TOK * ROWS) return;
  float s = 0.0f;
  if (live)
    for (int p = 0; p < WAVES; ++p) s += sums[(p * TOK + t) * 20 + i];
  if (has) {
    float d = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c * 8 < r)
#pragma unroll
        for (int e = 0; e < 8; ++e) d = fmaf(q[c][e], low[t * r + c * 8 + e], d);
    for (int k = 32; k < r; k += 8) {
      q[0].load(pb + k);
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fmaf(q[0][e], low[t * r + k + e], d);
    }
    s += d;
  }
  if (PAIR) {
    const float up = __shfl_xor(s, ROWS / 2);
    if (live && i < cols) out[(size_t)t * half + n0 + i] = float_to_bf16_bits(silu_f32(s) * up);
  } else if (live) {
    if (residual) s += bf16_bits_to_float(residual[(size_t)t * N + n0 + i]);
    out[(size_t)t * N + n0 + i] = float_to_bf16_bits(s);
  }
}

template <bool PAIR>
hipError_t small(const Ffn& f, const Lora& l, const void* x, int K, const void* w, int rows, const void* a,
                 const void* b, const float* scale, const int32_t* ids, const void* residual, void* out, void* ws,
                 hipStream_t st) {
  const Space s = space(f, l, ws);
  const int parts = parts_of(f, l, K);
  // Few low-rank values: every workgroup computes them for itself (two rows of A
  // a wave at most, from L2), which costs less than a launch.  One token,
  // rank 16, both projections: 12 us of kernels in two launches, 15 us in four (a
  // pass among others 16 and 24 us).
  const bool own = f.T * l.r <= 2 * stream_waves(16);
  if (!own) {
    hipLaunchKernelGGL((low_kernel<uint16_t, 4, false>), dim3(f.T * parts * (l.r / 4)), dim3(256), 0, st,
                       (const uint16_t*)x, (const uint16_t*)a, scale, ids, f.T, K, l.L, l.r, parts, s.v, s.perm,
                       s.sorted, s.first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  auto stream = [&](auto kernel, int per, int tokens) {
    hipLaunchKernelGGL(kernel, dim3(rows / per), dim3(stream_waves(tokens) * 64), 0, st, (const uint16_t*)x,
                       (const uint16_t*)w, (const uint16_t*)a, (const uint16_t*)b, scale, ids, s.v,
                       (const uint16_t*)residual, (uint16_t*)out, f.T, K, rows, l.L, l.r, parts);
    return hipGetLastError();
  };
  // sixteen rows a workgroup leave CUs without one below 4096 rows
  auto by_rows = [&](auto per) {
    constexpr int R = decltype(per)::value;
    if (f.T > 16) return stream(stream_kernel<PAIR, R, 32, false>, R, 32);
    return own ? stream(stream_kernel<PAIR, R, 16, true>, R, 16) : stream(stream_kernel<PAIR, R, 16, false>, R, 16);
  };
  return rows < 4096 ? by_rows(tile::Index<8>{}) : by_rows(tile::Index<16>{});
}

}  // namespace

size_t lora_workspace_bytes(const Ffn& f, const Lora& l) { return space(f, l, nullptr).bytes; }

hipError_t launch_lora_w13(const Ffn& f, const Lora& l, const void* x, const void* w1, const void* a, const void* b,
                           const float* scale, const int32_t* ids, void* hs, void* ws, hipStream_t st) {
  if (small_path(f)) return small<true>(f, l, x, f.H, w1, 2 * f.I, a, b, scale, ids, nullptr, hs, ws, st);
  if (f.bf16)
    return big<uint16_t>(f, l, x, f.H, w1, 2 * f.I, a, b, scale, ids, true, SwigluOut<uint16_t>{(uint16_t*)hs, f.I},
                         ws, st);
  return big<float>(f, l, x, f.H, w1, 2 * f.I, a, b, scale, ids, true, SwigluOut<float>{(float*)hs, f.I}, ws, st);
}

hipError_t launch_lora_down(const Ffn& f, const Lora& l, const void* hs, const void* w2, const void* a, const void* b,
                            const float* scale, const int32_t* ids, bool sorted, const void* residual, void* out,
                            void* ws, hipStream_t st) {
  if (small_path(f)) return small<false>(f, l, hs, f.I, w2, f.H, a, b, scale, ids, residual, out, ws, st);
  if (f.bf16)
    return big<uint16_t>(f, l, hs, f.I, w2, f.H, a, b, scale, ids, !sorted,
                         tile::StoreOut<uint16_t>{(uint16_t*)out, (const uint16_t*)residual, f.H}, ws, st);
  return big<float>(f, l, hs, f.I, w2, f.H, a, b, scale, ids, !sorted,
                    tile::StoreOut<float>{(float*)out, (const float*)residual, f.H}, ws, st);
}

}  // namespace moe
