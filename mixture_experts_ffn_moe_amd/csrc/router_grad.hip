// What the router is trained with: balance loss and per-expert counts, the
// gradient of the logits, of the routing weights, and of the router's weight.
// Formulas and argument semantics: moe_router_grad.h.
//
// Everything here streams its inputs once.  Sums over tokens run in a fixed
// order (per-workgroup partials in the workspace, then one summing pass), so
// no result depends on the order of atomics.
#include "../../include/moe_router_grad.h"
#include "api_check.h"
#include "lds_barrier.h"
#include "row_grid.h"

#include <algorithm>

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Softmax of four tokens per wave: 16 lanes per token, lane l of them holding
// experts l, l + 16, l + 32, l + 48.  A token then needs four-step reductions
// over 16 lanes, shared by the wave's four tokens (one token per wave, one
// lane per expert, would take six steps for each token alone).
constexpr int kTokWave = 4;
constexpr int kPer = kMaxExperts / 16;  // experts per lane

// Reduction over 16 lanes, the same bits in each of them: rotations within the
// row by 8, 4, 2 and 1 (DPP: no LDS round trip, of which a token would wait for
// sixteen in turn).
template <int CTRL, typename F>
__device__ __forceinline__ float row_step(float v, F f) {
  return f(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true)));
}
template <typename F>
__device__ __forceinline__ float row16_reduce(float v, F f) {
  v = row_step<0x128>(v, f);  // row_ror:8
  v = row_step<0x124>(v, f);
  v = row_step<0x122>(v, f);
  return row_step<0x121>(v, f);
}
__device__ __forceinline__ float row16_sum(float v) {
  return row16_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float row16_max(float v) {
  return row16_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

// e^x for x <= 0, to 2 units in the last place: 2^(x log2 e) with the product's
// rest as a first-order term.  0 below -87, where the result is subnormal; NaN
// stays NaN.  (Against expf, balance loss and gradient at T = 65535: 25 against 27 us.)
__device__ __forceinline__ float exp_nonpos(float x) {
  const float hi = 0x1.715476p+0f, lo = 0x1.4ae0bep-26f, ln2 = 0x1.62e430p-1f;  // hi + lo = log2 e
  const float t = x * hi;
  const float rest = fmaf(x, lo, fmaf(x, hi, -t));
  const float r = __builtin_amdgcn_exp2f(t);
  return x < -87.0f ? 0.0f : fmaf(r, rest * ln2, r);
}

// Probabilities of the token whose logits start at `row`, 0 past E and for a
// row that is not `ok` (its values are loaded from a valid address and dropped).
__device__ __forceinline__ void softmax16(const float (&v)[kPer], int l, int E, bool ok, float (&p)[kPer]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = fmaxf(m, l + 16 * i < E ? v[i] : -INFINITY);
  m = row16_max(m);
  if (m == -INFINITY) m = 0.0f;  // no finite logit: every exponential below is 0
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    p[i] = l + 16 * i < E ? exp_nonpos(v[i] - m) : 0.0f;
    s += p[i];
  }
  s = row16_sum(s);
  const float r = s > 0.0f ? 1.0f / s : 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) p[i] = ok ? p[i] * r : 0.0f;
}

// ---------------------------------------------------------------------------
// Balance loss.  One workgroup of 16 waves takes 64 tokens a step and a
// contiguous run of tokens in all; its sums go to the workspace in fp64, and
// a second launch of one workgroup adds them (one workgroup alone finishes by
// itself).  T = 4096, E = 64, k = 8: 5.0 + 2.7 us, launches; T = 65535: 8.0 - 9.5 +
// 5.0 us for 19 MB of logits and ids, the vector instructions of the softmax and two
// launches.
constexpr int kBalWaves = 16;
constexpr int kBalStep = kBalWaves * kTokWave;  // tokens per step of a workgroup
constexpr int kBalBlocks = 256;                 // at most one workgroup per CU

struct BalancePartial {
  double prob[kMaxExperts];
  int32_t count[kMaxExperts];
  int32_t valid;
  int32_t pad[15];
};

__device__ __forceinline__ void balance_write(double prob, int count, int n, int E, int k, int lane,
                                              int32_t* __restrict__ counts, float* __restrict__ mean_prob,
                                              float* __restrict__ loss) {
  const double mean = n > 0 ? prob / (double)n : 0.0;
  const double f = n > 0 ? (double)count / ((double)n * k) : 0.0;
  double s = lane < E ? f * mean : 0.0;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) s += __shfl_xor(s, d);
  if (lane < E) {
    counts[lane] = count;
    mean_prob[lane] = (float)mean;
  }
  if (lane == 0) loss[0] = (float)(E * s);
}

__global__ __launch_bounds__(kBalWaves * 64) void balance_partial(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int T,
    int E, int k, int per_block, BalancePartial* __restrict__ partial, int32_t* __restrict__ counts,
    float* __restrict__ mean_prob, float* __restrict__ loss) {
  __shared__ double prob[kBalWaves][kMaxExperts];
  __shared__ int hcnt[kMaxExperts + 1];  // counts, then the number of valid tokens
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int t_begin = blockIdx.x * per_block, t_end = min(T, t_begin + per_block);
  if (tid <= kMaxExperts) hcnt[tid] = 0;
  __syncthreads();

  double sum[kPer] = {};
  int valid = 0;
  // four steps' loads are in flight before the first is used (256 tokens, a
  // workgroup's share at 65536)
  constexpr int kAhead = 4;
  for (int t0 = t_begin; t0 < t_end; t0 += kAhead * kBalStep) {
    float v[kAhead][kPer];
    uint8_t mk[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int tc = min(t0 + u * kBalStep + wave * kTokWave + g, t_end - 1);
      mk[u] = mask != nullptr ? mask[tc] : (uint8_t)1;
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[u][i] = logits[(size_t)tc * E + min(l + 16 * i, E - 1)];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (t0 + u * kBalStep >= t_end) break;
      const bool ok = t0 + u * kBalStep + wave * kTokWave + g < t_end && mk[u] != 0;
      float p[kPer];
      softmax16(v[u], l, E, ok, p);
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum[i] += (double)p[i];
      valid += (ok && l == 0) ? 1 : 0;
    }
  }
  for (int r = t_begin * k + tid; r < t_end * k; r += kBalWaves * 64) {
    const int e = ids[r];
    if ((mask == nullptr || mask[r / k] != 0) && (unsigned)e < (unsigned)E) atomicAdd(&hcnt[e], 1);
  }
  // the wave's four tokens of a step, then the 16 waves, in a fixed order
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    double d = sum[i];
    d += __shfl_xor(d, 16);
    d += __shfl_xor(d, 32);
    if (g == 0) prob[wave][l + 16 * i] = d;
  }
  if (l == 0 && valid > 0) atomicAdd(&hcnt[kMaxExperts], valid);
  __syncthreads();
  if (wave != 0) return;
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kBalWaves; ++w) s += prob[w][lane];
  if (gridDim.x == 1) {
    balance_write(s, hcnt[lane], hcnt[kMaxExperts], E, k, lane, counts, mean_prob, loss);
    return;
  }
  BalancePartial& out = partial[blockIdx.x];
  out.prob[lane] = s;
  out.count[lane] = hcnt[lane];
  if (lane == 0) out.valid = hcnt[kMaxExperts];
}

__global__ __launch_bounds__(kBalWaves * 64) void balance_finish(const BalancePartial* __restrict__ partial, int nb,
                                                                 int E, int k, int32_t* __restrict__ counts,
                                                                 float* __restrict__ mean_prob,
                                                                 float* __restrict__ loss) {
  __shared__ double prob[kBalWaves][kMaxExperts];
  __shared__ int cnt[kBalWaves][kMaxExperts], val[kBalWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double s = 0.0;
  int c = 0, n = 0;
  for (int b = wave; b < nb; b += 4 * kBalWaves) {  // four partials in flight
    double pv[4];
    int cv[4], nv[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const BalancePartial& q = partial[min(b + u * kBalWaves, nb - 1)];
      pv[u] = q.prob[lane];
      cv[u] = q.count[lane];
      nv[u] = q.valid;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool in = b + u * kBalWaves < nb;
      s += in ? pv[u] : 0.0;
      c += in ? cv[u] : 0;
      n += in ? nv[u] : 0;
    }
  }
  prob[wave][lane] = s;
  cnt[wave][lane] = c;
  if (lane == 0) val[wave] = n;
  __syncthreads();
  if (wave != 0) return;
  s = 0.0;
  c = 0;
  n = 0;
#pragma unroll
  for (int w = 0; w < kBalWaves; ++w) {
    s += prob[w][lane];
    c += cnt[w][lane];
    n += val[w];
  }
  balance_write(s, c, n, E, k, lane, counts, mean_prob, loss);
}

// ---------------------------------------------------------------------------
// Gradient of the logits: 16 lanes per token as above.  The routes' values
// are scattered to the experts through an LDS row per token (written and read
// by the token's own wave).  T = 4096, E = 64, k = 8: 4.3 us; T = 65535: 11.6 us
// for 40 MB (3.4 TB/s).
constexpr int kRbWaves = 4;

__global__ __launch_bounds__(kRbWaves * 64) void route_backward(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ topw,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts, const float* __restrict__ d_w,
    const float* __restrict__ d_loss, int T, int E, int k, int renorm, float* __restrict__ d_logits) {
  __shared__ float sel[kRbWaves][kTokWave][kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane & 15, g = lane >> 4;
  float* row = sel[wave][g];

  // f[e] of this lane's experts and the loss's coefficient d_loss * E / N
  float f[kPer] = {}, coef = 0.0f;
  if (d_loss != nullptr) {
    const int ce = lane < E ? counts[lane] : 0;
    int total = ce;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) total += __shfl_xor(total, d);
    const float fe = total > 0 ? (float)((double)ce / (double)total) : 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) f[i] = __shfl(fe, l + 16 * i);
    coef = total > 0 ? (float)((double)d_loss[0] * E * k / (double)total) : 0.0f;
  }
  const bool need_p = d_loss != nullptr || !renorm;

  for (int t0 = blockIdx.x * kRbWaves * kTokWave; t0 < T; t0 += gridDim.x * kRbWaves * kTokWave) {
    const int t = t0 + wave * kTokWave + g;
    const int tc = min(t, T - 1);
    const bool ok = t < T && (mask == nullptr || mask[tc] != 0);
    float p[kPer] = {}, d[kPer] = {};
    // the first 16 routes' values beside the logits (k is 8, mostly); more of
    // them are read again below
    const size_t r0 = (size_t)tc * k + min(l, k - 1);
    float w0 = 0.0f, dw0 = 0.0f, v[kPer] = {};
    int e0 = -1;
    if (need_p) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = logits[(size_t)tc * E + min(l + 16 * i, E - 1)];
    }
    if (d_w != nullptr) {
      w0 = topw[r0];
      dw0 = d_w[r0];
      e0 = ids[r0];
    }
    if (need_p) {
      softmax16(v, l, E, ok, p);
      float fp = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) fp = fmaf(f[i], p[i], fp);
      fp = row16_sum(fp);
#pragma unroll
      for (int i = 0; i < kPer; ++i) d[i] = coef * p[i] * (f[i] - fp);
    }
    if (d_w != nullptr) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) row[l + 16 * i] = 0.0f;
      float dot = l < k ? w0 * dw0 : 0.0f;
      for (int j = l + 16; j < k; j += 16) {
        const size_t r = (size_t)tc * k + j;
        dot = fmaf(topw[r], d_w[r], dot);
      }
      dot = row16_sum(dot);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (l < k && (unsigned)e0 < (unsigned)E) row[e0] = renorm ? w0 * (dw0 - dot) : dw0;
      for (int j = l + 16; j < k; j += 16) {
        const size_t r = (size_t)tc * k + j;
        const int e = ids[r];
        if ((unsigned)e < (unsigned)E) row[e] = renorm ? topw[r] * (d_w[r] - dot) : d_w[r];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float s = row[l + 16 * i];
        d[i] += renorm ? s : p[i] * (s - dot);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    if (t < T) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (l + 16 * i < E) d_logits[(size_t)t * E + l + 16 * i] = ok ? d[i] : 0.0f;
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient of the routing weights: one workgroup per token, as the finalize
// whose backward pass it is; d_out's row is read once per eight routes, each
// thread taking 8 columns (inside one y block) of d_out and of eight rows of y.
// Bound by HBM: T = 4096, H = 4096, k = 8, bf16: 302 MB in 54 us (5.6 TB/s); fp32,
// T = 1024: 134 MB in 28 us at k = 8, 67 MB in 15 us at k = 4.
constexpr int kFbThreads = 256;
constexpr int kFbRoutes = 8;

__device__ __forceinline__ void load_cols8(const uint16_t* p, float (&v)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load_cols8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// dot of 8 columns of one y row with d
__device__ __forceinline__ float ydot8(const float* y, const int8_t*, size_t row, int H, int c, const float (&d)[8]) {
  float v[8], s = 0.0f;
  load_cols8(y + row * H + c, v);
#pragma unroll
  for (int q = 0; q < 8; ++q) s = fmaf(v[q], d[q], s);
  return s;
}
__device__ __forceinline__ float ydot8(const _Float16* y, const int8_t* ye, size_t row, int H, int c,
                                       const float (&d)[8]) {
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  const f16x8 h = *reinterpret_cast<const f16x8*>(y + row * H + c);
  const int e = ye[row * ((H + kYBlock - 1) / kYBlock) + c / kYBlock];
  float s = 0.0f;
#pragma unroll
  for (int q = 0; q < 8; ++q) s = fmaf((float)h[q], d[q], s);
  return ldexpf(s, e);
}

// NJ routes [j0, j0 + NJ) of token t (NJ known to the compiler: the NJ row
// loads of a step are all in flight before the first is used; of fp32 rows at NJ = 8
// it takes one row's loads at a time, to which the other workgroups of a CU
// give cover: 4.8 TB/s, and 4.5 at NJ = 4).
template <int NJ, typename T, typename YT>
__device__ __forceinline__ void finalize_backward_routes(const YT* __restrict__ y, const int8_t* __restrict__ ye,
                                                         const int32_t* __restrict__ inv,
                                                         const T* __restrict__ d_out, int H,
                                                         float (&part)[kFbThreads / 64][kFbRoutes],
                                                         float* __restrict__ d_w) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  size_t rows[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) rows[j] = (size_t)inv[j];
  float acc[NJ] = {};
  for (int c = tid * 8; c < H; c += kFbThreads * 8) {
    float d[8];
    load_cols8(d_out + c, d);
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] += ydot8(y, ye, rows[j], H, c, d);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) acc[j] += __shfl_xor(acc[j], s);
    if (lane == 0) part[wave][j] = acc[j];
  }
  __syncthreads();
  if (tid < NJ) {
    float s = part[0][tid];
#pragma unroll
    for (int w = 1; w < kFbThreads / 64; ++w) s += part[w][tid];
    d_w[tid] = s;
  }
  __syncthreads();
}

template <typename T, typename YT>
__global__ __launch_bounds__(kFbThreads) void finalize_backward(const YT* __restrict__ y,
                                                                const int8_t* __restrict__ ye,
                                                                const int32_t* __restrict__ inv,
                                                                const T* __restrict__ d_out, int tokens, int H,
                                                                int k, float* __restrict__ d_w) {
  __shared__ float part[kFbThreads / 64][kFbRoutes];
  const int t = grid_row();
  if (t >= tokens) return;
  inv += (size_t)t * k;
  d_w += (size_t)t * k;
  d_out += (size_t)t * H;
  int j = 0;
  for (; j + 8 <= k; j += 8) finalize_backward_routes<8>(y, ye, inv + j, d_out, H, part, d_w + j);
  if (k & 4) {
    finalize_backward_routes<4>(y, ye, inv + j, d_out, H, part, d_w + j);
    j += 4;
  }
  if (k & 2) {
    finalize_backward_routes<2>(y, ye, inv + j, d_out, H, part, d_w + j);
    j += 2;
  }
  if (k & 1) finalize_backward_routes<1>(y, ye, inv + j, d_out, H, part, d_w + j);
}

// ---------------------------------------------------------------------------
// Gradient of the router's weight, fp32 x, on v_mfma_f32_16x16x4_f32: a lane supplies
// one token's (k = lane/16) d_logits of expert 16 mt + lane%16 as A and one
// token's x column as B, so both operands are taken as they lie in memory.  A
// lane loads four neighbouring columns 4 (lane%16) + q; column tile q then
// holds columns q, q + 4, ..., and a lane's four results of a row are
// neighbours again.  A workgroup covers 64 experts x 64 columns over one run
// of tokens, its 16 waves taking every 16th step of 4 tokens; the waves' sums
// are added through LDS in a fixed order.  T = 4096, H = 4096: 41 us for 67 MB, the
// matrix instructions 14 of them.  Bound by latency: the compiler makes the loads of
// d_logits conditional and waits for each, nothing is asked for ahead (the bf16 kernel
// below is rid of that by bounded loads).
typedef float f32x4v __attribute__((ext_vector_type(4)));
constexpr int kWgWaves = 16;
constexpr int kWgCols = 64;
constexpr int kWgBlocks = 256;    // workgroups aimed at
constexpr int kWgMinTokens = 64;  // fewest tokens worth a workgroup of their own

inline int wgrad_splits(int T, int H) {
  return std::max(1, std::min(kWgBlocks / (H / kWgCols), (T + kWgMinTokens - 1) / kWgMinTokens));
}

// part: [splits][64][H] then [splits][64] bias sums; one split writes the results themselves
__global__ __launch_bounds__(kWgWaves * 64) void router_weight_grad(
    const float* __restrict__ x, const float* __restrict__ dl, const uint8_t* __restrict__ mask, int T, int H, int E,
    int per_split, float* __restrict__ part, float* __restrict__ bias_part, float* __restrict__ d_wg,
    float* __restrict__ d_bias) {
  __shared__ float red[kWgWaves / 2][kMaxExperts][kWgCols];
  __shared__ float bred[kWgWaves][kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int split = blockIdx.y, h0 = blockIdx.x * kWgCols;
  const int t_begin = split * per_split, t_end = min(T, t_begin + per_split);
  f32x4v acc[4][4];
  float bsum[4] = {};
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[m][q] = f32x4v{0.f, 0.f, 0.f, 0.f};

  for (int t0 = t_begin + wave * 4; t0 < t_end; t0 += kWgWaves * 4) {
    const int t = t0 + g, tc = min(t, t_end - 1);
    const bool ok = t < t_end && (mask == nullptr || mask[tc] != 0);
    f32x4v b = *reinterpret_cast<const f32x4v*>(x + (size_t)tc * H + h0 + 4 * l);
    float a[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int e = 16 * m + l;
      const float v = dl[(size_t)tc * E + min(e, E - 1)];
      a[m] = ok && e < E ? v : 0.0f;
      bsum[m] += a[m];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) b[q] = ok ? b[q] : 0.0f;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[m][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[m], b[q], acc[m][q], 0, 0, 0);
  }
  // D layout: register r of a lane holds row 4 (lane/16) + r, column lane%16
#pragma unroll
  for (int half = kWgWaves / 2; half >= 1; half >>= 1) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<f32x4v*>(&red[wave - half][16 * m + 4 * g + r][4 * l]) =
              f32x4v{acc[m][0][r], acc[m][1][r], acc[m][2][r], acc[m][3][r]};
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4v o = *reinterpret_cast<const f32x4v*>(&red[wave][16 * m + 4 * g + r][4 * l]);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[m][q][r] += o[q];
        }
    }
    __syncthreads();
  }
  const bool last = gridDim.y == 1;
  if (wave == 0) {
    float* out = last ? d_wg : part + (size_t)split * kMaxExperts * H;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int e = 16 * m + 4 * g + r;
        if (e < E)
          *reinterpret_cast<f32x4v*>(out + (size_t)e * H + h0 + 4 * l) =
              f32x4v{acc[m][0][r], acc[m][1][r], acc[m][2][r], acc[m][3][r]};
      }
  }
  if (blockIdx.x != 0) return;
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    float v = bsum[m];
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    if (g == 0) bred[wave][16 * m + l] = v;
  }
  __syncthreads();
  if (tid < kMaxExperts) {
    float s = bred[0][tid];
#pragma unroll
    for (int w = 1; w < kWgWaves; ++w) s += bred[w][tid];
    if (!last)
      bias_part[split * kMaxExperts + tid] = s;
    else if (d_bias != nullptr && tid < E)
      d_bias[tid] = s;
  }
}

// The same for bf16 x on v_mfma_f32_16x16x32_bf16.  d_logits enter as three
// bf16 parts (the upper 8 bits of the significand, the next 8, the last 8:
// each difference is exact), so a product is as exact as in fp32 at 3/16 of
// the fp32 matrix time.  A workgroup of 8 waves takes CG x 64 columns and, per
// step, TG x 32 tokens (CG TG = 8), a wave 64 columns of 32 tokens.
// d_logits of a step are cut once per workgroup, by all of its threads, and
// passed through LDS in operand order, one step ahead.  (Cut by every wave
// for itself, the vector instructions took most of the time: 183 against 81 us
// at 32767 tokens when that was changed.)  x wants a lane to hold 8 tokens of one column and lies in
// memory token by token: a lane loads four neighbouring columns of its 8
// tokens and puts pairs of tokens together with byte permutations; column tile
// c then holds columns 4 (lane%16) + c.
// Small CG means few partial sums (a workgroup writes 64 experts x its columns),
// large CG that d_logits are cut and read less often.  CG = 2 against 4, both
// launches with a mask (without one CG = 4 gains a little less), us:
//   H = 1024: T = 16384 31 / 39, 65536 56 / 61, 98304 79 / 74, 262144 172 / 158
//   H = 2048: T = 16384 33 / 34, 49152 65 / 64, 131071 157 / 147
//   H = 4096: T = 4096 21 / 24, 16384 46 / 46, 24576 62 / 60, 65535 152 / 140
//   H = 8192: T = 4096 29 / 30, 16384 77 / 73, 65535 288 / 261
// and of narrower x, whose few columns CG = 4 leaves to few waves, H = 64: T =
// 1572864 186 / 252, H = 256: 393216 104 / 132, H = 512: 196608 87 / 92, 1048576
// 325 / 307.  Bound by the chain of a step, load to cut to product, with two waves
// a SIMD (268 MB of x in 71 us: 3.8 TB/s).
constexpr int kWbWaves = 8;
constexpr int kWbTok = 32;  // tokens of a wave's step

inline int wgrad_groups(int T, int H) { return H >= 512 && (long long)T * H >= 3 << 25 ? 4 : 2; }
inline int wgrad_bf16_splits(int T, int H) {
  const int cg = wgrad_groups(T, H), cols = (H / kWgCols + cg - 1) / cg, step = kWbWaves / cg * kWbTok;
  return std::max(1, std::min(kWgBlocks / cols, (T + 2 * step - 1) / (2 * step)));
}

// the upper halves of two words, and the lower halves
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }
__device__ __forceinline__ uint32_t pack_lo(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }

template <int CG, bool MASK>
__global__ __launch_bounds__(kWbWaves * 64) void router_weight_grad_bf16(
    const uint16_t* __restrict__ x, const float* __restrict__ dl, const uint8_t* __restrict__ mask, int T, int H,
    int E, int per_split, float* __restrict__ part, float* __restrict__ bias_part, float* __restrict__ d_wg,
    float* __restrict__ d_bias) {
  constexpr int TG = kWbWaves / CG;
  constexpr int kStep = TG * kWbTok;              // tokens of a step
  constexpr int kPieces = kStep / 8 / kWbWaves;   // (8 tokens of one expert) that a thread cuts per step
  constexpr int kBuf = TG * 3 * 4 * 1024;         // [token group][part][expert tile][lane] x 16 bytes
  constexpr int kRed = TG / 2 * CG * kMaxExperts * kWgCols * 4;  // the final sums, which reuse the buffers
  __shared__ __attribute__((aligned(1024))) char lds[2 * kBuf > kRed ? 2 * kBuf : kRed];
  __shared__ float bred[kWbWaves][kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l = lane & 15, g = lane >> 4;
  const int cg = wave % CG, tg = wave / CG;
  const int split = blockIdx.y;
  const int hc = blockIdx.x * CG + cg;            // column group; past the last it repeats it and stores nothing
  const int h0 = min(hc, H / kWgCols - 1) * kWgCols;
  const int t_begin = split * per_split, t_end = min(T, t_begin + per_split);

  // Loads are bounded by the hardware and never conditional: rows from t_end on
  // return zeros without touching memory.  (With branches for the last tokens the
  // compiler waits for every load in flight before it uses one: 87 against 77 us
  // at 32767 tokens, 20 against 16 at 4096.)
  // n tokens from t on, rows of `bytes`: their resource.
  auto tokens = [&](const void* p, size_t bytes, int t, int n) {
    const char* at = uniform_ptr((const char*)p + (size_t)min(t, T) * bytes);
    const uint32_t size = (uint32_t)((size_t)max(0, min(t_end - t, n)) * bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), 0, __builtin_amdgcn_readfirstlane((int)size), 0x00020000);
  };

  // d_logits of a step: thread (wave, lane) takes expert `lane` of the tokens
  // 8 (wave + 8 j) .. + 7; experts past E lie out of bounds too
  struct Cut {
    float v[kPieces][8];
    uint8_t ok[kPieces];  // of token lane % 8, as loaded: decoding waits for the load
  };
  const uint32_t d_off = lane < E ? lane * 4u : 0x7ffff000u;
  auto load_d = [&](int t0, Cut& b) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int tb = t0 + 8 * (wave + kWbWaves * j);
      if constexpr (MASK) b.ok[j] = mask[min(tb + (lane & 7), T - 1)];
      const auto rows = tokens(dl, (size_t)E * 4, tb, 8);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        b.v[j][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rows, d_off + (uint32_t)(i * E) * 4u, 0, 0));
    }
  };
  float bsum = 0.0f;
  auto cut_d = [&](const Cut& b, int buf) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int pc = wave + kWbWaves * j;
      const uint32_t ok = MASK ? (uint32_t)__ballot(b.ok[j] != 0) : ~0u;
      float v[8], r1[8], r2[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = (ok >> i & 1) != 0 ? b.v[j][i] : 0.0f;
        bsum += v[i];
        r1[i] = v[i] - __uint_as_float(__float_as_uint(v[i]) & 0xffff0000u);
        r2[i] = r1[i] - __uint_as_float(__float_as_uint(r1[i]) & 0xffff0000u);
      }
      char* at = lds + buf * kBuf + (pc / 4 * 12 + lane / 16) * 1024 + (pc % 4 * 16 + lane % 16) * 16;
      auto pack8 = [](const float (&f)[8]) {
        return make_uint4(pack_hi(__float_as_uint(f[0]), __float_as_uint(f[1])),
                          pack_hi(__float_as_uint(f[2]), __float_as_uint(f[3])),
                          pack_hi(__float_as_uint(f[4]), __float_as_uint(f[5])),
                          pack_hi(__float_as_uint(f[6]), __float_as_uint(f[7])));
      };
      *reinterpret_cast<uint4*>(at) = pack8(v);
      *reinterpret_cast<uint4*>(at + 4096) = pack8(r1);
      *reinterpret_cast<uint4*>(at + 8192) = pack8(r2);
    }
  };
  // x of this wave's tokens of a step
  struct Rows {
    uint2 v[8];
    uint8_t ok;  // of token lane % 32
  };
  const uint32_t x_off = ((uint32_t)(8 * g) * (uint32_t)H + (uint32_t)(h0 + 4 * l)) * 2u;
  auto load_x = [&](int t0, Rows& b) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const int tw = t0 + tg * kWbTok;
    if constexpr (MASK) b.ok = mask[min(tw + (lane & 31), T - 1)];
    const auto rows = tokens(x, (size_t)H * 2, tw, kWbTok);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rows, x_off + (uint32_t)i * (uint32_t)H * 2u, 0, 0);
      b.v[i] = make_uint2(v.x, v.y);
    }
  };

  f32x4v acc[4][4];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[m][c] = f32x4v{0.f, 0.f, 0.f, 0.f};

  auto products = [&](Rows& b, int buf) {
    if constexpr (MASK) {
      const uint32_t bits = (uint32_t)__ballot(b.ok != 0);
      if (bits != ~0u) {  // rows that do not count may hold anything
        const uint32_t mine = bits >> (8 * g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool ok = (mine >> i & 1) != 0;
          b.v[i] = make_uint2(ok ? b.v[i].x : 0u, ok ? b.v[i].y : 0u);
        }
      }
    }
    bf16x8 bx[4];  // column tile c
    bx[0] = __builtin_bit_cast(bf16x8, make_uint4(pack_lo(b.v[0].x, b.v[1].x), pack_lo(b.v[2].x, b.v[3].x),
                                                  pack_lo(b.v[4].x, b.v[5].x), pack_lo(b.v[6].x, b.v[7].x)));
    bx[1] = __builtin_bit_cast(bf16x8, make_uint4(pack_hi(b.v[0].x, b.v[1].x), pack_hi(b.v[2].x, b.v[3].x),
                                                  pack_hi(b.v[4].x, b.v[5].x), pack_hi(b.v[6].x, b.v[7].x)));
    bx[2] = __builtin_bit_cast(bf16x8, make_uint4(pack_lo(b.v[0].y, b.v[1].y), pack_lo(b.v[2].y, b.v[3].y),
                                                  pack_lo(b.v[4].y, b.v[5].y), pack_lo(b.v[6].y, b.v[7].y)));
    bx[3] = __builtin_bit_cast(bf16x8, make_uint4(pack_hi(b.v[0].y, b.v[1].y), pack_hi(b.v[2].y, b.v[3].y),
                                                  pack_hi(b.v[4].y, b.v[5].y), pack_hi(b.v[6].y, b.v[7].y)));
    const char* frag = lds + buf * kBuf + tg * 12 * 1024 + (g * 16 + l) * 16;
#pragma unroll
    for (int q = 2; q >= 0; --q)  // smallest part first
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(frag + (q * 4 + m) * 1024);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, bx[c], acc[m][c], 0, 0, 0);
      }
  };
  // Step s: its x and cut d_logits are here; the next step's d_logits are cut
  // meanwhile.  x is asked for two steps ahead, d_logits three.  (x four steps
  // ahead, in twice the registers: 73 against 76 us at 32767 tokens, 19 against
  // 16 at 4096.)
  const int steps = t_end > t_begin ? (t_end - t_begin + kStep - 1) / kStep : 0;
  if (steps > 0) {
    Rows xr[2];
    Cut dr[2];
    auto at = [&](int s) { return t_begin + s * kStep; };  // past the last step: nothing is loaded
    load_d(at(0), dr[0]);
    load_d(at(1), dr[1]);
    load_x(at(0), xr[0]);
    load_x(at(1), xr[1]);
    __builtin_amdgcn_sched_barrier(0);
    cut_d(dr[0], 0);
    load_d(at(2), dr[0]);
    lds_barrier();
    auto step = [&](int s, Rows& cur, Cut& d) {
      products(cur, s & 1);
      cut_d(d, (s + 1) & 1);  // past the last step: zeros
      load_d(at(s + 3), d);  // first: loads return in order, and these are waited for first
      load_x(at(s + 2), cur);
      __builtin_amdgcn_sched_barrier(0);
      lds_barrier();
    };
    for (int s = 0; s < steps; s += 2) {  // one step of zeros more if they are odd
      step(s, xr[0], dr[1]);
      step(s + 1, xr[1], dr[0]);
    }
  }

  // D layout: register r of a lane holds row 4 g + r of the expert tile, column l of the column tile
  float(*red)[kMaxExperts][kWgCols] = reinterpret_cast<float(*)[kMaxExperts][kWgCols]>(lds);
#pragma unroll
  for (int half = TG / 2; half >= 1; half >>= 1) {
    if (tg >= half && tg < 2 * half) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<f32x4v*>(&red[(tg - half) * CG + cg][16 * m + 4 * g + r][4 * l]) =
              f32x4v{acc[m][0][r], acc[m][1][r], acc[m][2][r], acc[m][3][r]};
    }
    __syncthreads();
    if (tg < half) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4v o = *reinterpret_cast<const f32x4v*>(&red[tg * CG + cg][16 * m + 4 * g + r][4 * l]);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[m][c][r] += o[c];
        }
    }
    __syncthreads();
  }
  const bool last = gridDim.y == 1;
  if (tg == 0 && hc < H / kWgCols) {
    float* out = last ? d_wg : part + (size_t)split * kMaxExperts * H;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (16 * m + 4 * g + r < E)
          *reinterpret_cast<f32x4v*>(out + (size_t)(16 * m + 4 * g + r) * H + h0 + 4 * l) =
              f32x4v{acc[m][0][r], acc[m][1][r], acc[m][2][r], acc[m][3][r]};
  }
  if (blockIdx.x != 0) return;
  bred[wave][lane] = bsum;
  __syncthreads();
  if (tid < kMaxExperts) {
    float s = bred[0][tid];
#pragma unroll
    for (int w = 1; w < kWbWaves; ++w) s += bred[w][tid];
    if (!last)
      bias_part[split * kMaxExperts + tid] = s;
    else if (d_bias != nullptr && tid < E)
      d_bias[tid] = s;
  }
}

// Sum of the splits, ascending; one thread per four columns.
__global__ __launch_bounds__(256) void router_weight_sum(const float* __restrict__ part,
                                                         const float* __restrict__ bias_part, int splits, int H,
                                                         int E, float* __restrict__ d_wg, float* __restrict__ d_bias) {
  const int i = blockIdx.x * 256 + threadIdx.x, n4 = E * H / 4;
  if (i < n4) {
    f32x4v s = f32x4v{0.f, 0.f, 0.f, 0.f};
    int p = 0;
    for (; p + 4 <= splits; p += 4) {  // four loads in flight
      f32x4v v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = reinterpret_cast<const f32x4v*>(part + (size_t)(p + u) * kMaxExperts * H)[i];
#pragma unroll
      for (int u = 0; u < 4; ++u) s += v[u];
    }
    for (; p < splits; ++p) s += reinterpret_cast<const f32x4v*>(part + (size_t)p * kMaxExperts * H)[i];
    reinterpret_cast<f32x4v*>(d_wg)[i] = s;
  }
  if (d_bias != nullptr && blockIdx.x == 0 && threadIdx.x < E) {
    float s = 0.0f;
    for (int p = 0; p < splits; ++p) s += bias_part[p * kMaxExperts + threadIdx.x];
    d_bias[threadIdx.x] = s;
  }
}

// T == 0: the sums over no tokens.
__global__ __launch_bounds__(256) void zero_words(uint32_t* a, size_t na, uint32_t* b, size_t nb, uint32_t* c,
                                                  size_t nc) {
  const size_t i = blockIdx.x * (size_t)256 + threadIdx.x;
  if (i < na) a[i] = 0u;
  if (b != nullptr && i < nb) b[i] = 0u;
  if (c != nullptr && i < nc) c[i] = 0u;
}

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

inline int balance_blocks(int T) { return std::max(1, std::min(kBalBlocks, ceil_div(T, kBalStep))); }

inline size_t wgrad_workspace(const Shape& s) {
  const size_t sp = (size_t)(s.bf16 ? wgrad_bf16_splits(s.T, s.H) : wgrad_splits(s.T, s.H));
  return sp == 1 ? 256 : sp * kMaxExperts * ((size_t)s.H + 1) * 4;
}

}  // namespace
}  // namespace moe

using namespace moe_api;

namespace {

moe_status check_workspace(const void* workspace, size_t have, size_t need) {
  if (workspace == nullptr || have < need) return MOE_ERR_WORKSPACE;
  if (((uintptr_t)workspace & (kAlign - 1)) != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_balance_workspace_size(const moe_shape* shape) {
  Shape s;
  if (check_shape(shape, &s) != MOE_OK) return 0;
  return align_up((size_t)moe::balance_blocks(s.T) * sizeof(moe::BalancePartial));
}

moe_status moe_balance_loss(const moe_shape* shape, const float* logits, const int32_t* topk_ids,
                            const uint8_t* token_mask, int32_t* counts, float* mean_prob, float* loss,
                            void* workspace, size_t workspace_bytes, void* stream) {
  Shape s;
  MOE_CHECK(check_shape(shape, &s));
  MOE_CHECK(check_ptr(counts)); MOE_CHECK(check_ptr(mean_prob)); MOE_CHECK(check_ptr(loss));
  hipStream_t st = (hipStream_t)stream;
  if (s.T == 0) {
    hipLaunchKernelGGL(moe::zero_words, dim3(1), dim3(256), 0, st, (uint32_t*)counts, (size_t)s.E,
                       (uint32_t*)mean_prob, (size_t)s.E, (uint32_t*)loss, (size_t)1);
    return hip_status(hipGetLastError());
  }
  MOE_CHECK(check_ptr(logits)); MOE_CHECK(check_ptr(topk_ids));
  if (token_mask != nullptr) MOE_CHECK(check_ptr(token_mask));
  MOE_CHECK(check_workspace(workspace, workspace_bytes, moe_balance_workspace_size(shape)));
  const int nb = moe::balance_blocks(s.T);
  moe::BalancePartial* part = (moe::BalancePartial*)workspace;
  hipLaunchKernelGGL(moe::balance_partial, dim3(nb), dim3(moe::kBalWaves * 64), 0, st, logits, topk_ids, token_mask,
                     s.T, s.E, s.k, moe::ceil_div(s.T, nb), part, counts, mean_prob, loss);
  if (nb > 1)
    hipLaunchKernelGGL(moe::balance_finish, dim3(1), dim3(moe::kBalWaves * 64), 0, st, part, nb, s.E, s.k, counts,
                       mean_prob, loss);
  return hip_status(hipGetLastError());
}

moe_status moe_route_backward(const moe_shape* shape, const float* logits, const int32_t* topk_ids,
                              const float* topk_w, const uint8_t* token_mask, const int32_t* counts,
                              const float* d_topk_w, const float* d_loss, float* d_logits, void* stream) {
  Shape s;
  MOE_CHECK(check_shape(shape, &s));
  if (s.T == 0) return MOE_OK;
  if (d_topk_w == nullptr && d_loss == nullptr) return MOE_ERR_INVALID_ARG;
  MOE_CHECK(check_ptr(logits)); MOE_CHECK(check_ptr(d_logits));
  if (token_mask != nullptr) MOE_CHECK(check_ptr(token_mask));
  if (d_topk_w != nullptr) {
    MOE_CHECK(check_ptr(d_topk_w)); MOE_CHECK(check_ptr(topk_ids)); MOE_CHECK(check_ptr(topk_w));
  }
  if (d_loss != nullptr) { MOE_CHECK(check_ptr(d_loss)); MOE_CHECK(check_ptr(counts)); }
  const int blocks = std::min(2048, moe::ceil_div(s.T, moe::kRbWaves * moe::kTokWave));
  hipLaunchKernelGGL(moe::route_backward, dim3(blocks), dim3(moe::kRbWaves * 64), 0, (hipStream_t)stream, logits,
                     topk_ids, topk_w, token_mask, counts, d_topk_w, d_loss, s.T, s.E, s.k, (int)s.renorm, d_logits);
  return hip_status(hipGetLastError());
}

size_t moe_router_grad_workspace_size(const moe_shape* shape) {
  Shape s;
  if (check_shape(shape, &s) != MOE_OK) return 0;
  return align_up(moe::wgrad_workspace(s));
}

moe_status moe_router_weight_grad(const moe_shape* shape, const void* x, const float* d_logits,
                                  const uint8_t* token_mask, float* d_wg, float* d_bias, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  Shape s;
  MOE_CHECK(check_shape(shape, &s));
  MOE_CHECK(check_ptr(d_wg));
  if (d_bias != nullptr) MOE_CHECK(check_ptr(d_bias));
  hipStream_t st = (hipStream_t)stream;
  if (s.T == 0) {
    const size_t n = (size_t)s.E * s.H;
    hipLaunchKernelGGL(moe::zero_words, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, (uint32_t*)d_wg, n,
                       (uint32_t*)d_bias, (size_t)s.E, (uint32_t*)nullptr, (size_t)0);
    return hip_status(hipGetLastError());
  }
  MOE_CHECK(check_ptr(x)); MOE_CHECK(check_ptr(d_logits));
  if (token_mask != nullptr) MOE_CHECK(check_ptr(token_mask));
  MOE_CHECK(check_workspace(workspace, workspace_bytes, moe_router_grad_workspace_size(shape)));
  const int splits = s.bf16 ? moe::wgrad_bf16_splits(s.T, s.H) : moe::wgrad_splits(s.T, s.H);
  int per = moe::ceil_div(s.T, splits);
  float* part = (float*)workspace;
  float* bpart = part + (size_t)splits * moe::kMaxExperts * s.H;
  if (s.bf16) {
    const int cg = moe::wgrad_groups(s.T, s.H);
    const dim3 grid(moe::ceil_div(s.H / moe::kWgCols, cg), splits);
    per = moe::ceil_div(per, moe::kWbTok) * moe::kWbTok;
#define MOE_GO(CG, MASK)                                                                                           \
  hipLaunchKernelGGL((moe::router_weight_grad_bf16<CG, MASK>), grid, dim3(moe::kWbWaves * 64), 0, st,              \
                     (const uint16_t*)x, d_logits, token_mask, s.T, s.H, s.E, per, part, bpart, d_wg, d_bias)
    if (cg == 4 && token_mask != nullptr) MOE_GO(4, true);
    else if (cg == 4) MOE_GO(4, false);
    else if (token_mask != nullptr) MOE_GO(2, true);
    else MOE_GO(2, false);
#undef MOE_GO
  } else {
    hipLaunchKernelGGL(moe::router_weight_grad, dim3(s.H / moe::kWgCols, splits), dim3(moe::kWgWaves * 64), 0, st, (const float*)x, d_logits,
                       token_mask, s.T, s.H, s.E, per, part, bpart, d_wg, d_bias);
  }
  if (splits > 1)
    hipLaunchKernelGGL(moe::router_weight_sum, dim3(moe::ceil_div(s.E * s.H / 4, 256)), dim3(256), 0, st, part, bpart,
                       splits, s.H, s.E, d_wg, d_bias);
  return hip_status(hipGetLastError());
}

moe_status moe_finalize_backward(const moe_shape* shape, const void* y, const int32_t* inv, const void* d_out,
                                 float* d_topk_w, void* stream) {
  Shape s;
  MOE_CHECK(check_shape(shape, &s));
  if (s.T == 0) return MOE_OK;
  MOE_CHECK(check_ptr(y)); MOE_CHECK(check_ptr(inv)); MOE_CHECK(check_ptr(d_out)); MOE_CHECK(check_ptr(d_topk_w));
  hipStream_t st = (hipStream_t)stream;
  if (s.bf16)
    hipLaunchKernelGGL((moe::finalize_backward<uint16_t, _Float16>), moe::row_grid(s.T), dim3(moe::kFbThreads), 0, st,
                       (const _Float16*)y, (const int8_t*)y + (size_t)s.R() * s.H * 2, inv, (const uint16_t*)d_out,
                       s.T, s.H, s.k, d_topk_w);
  else
    hipLaunchKernelGGL((moe::finalize_backward<float, float>), moe::row_grid(s.T), dim3(moe::kFbThreads), 0, st,
                       (const float*)y, (const int8_t*)nullptr, inv, (const float*)d_out, s.T, s.H, s.k, d_topk_w);
  return hip_status(hipGetLastError());
}

}  // extern "C"
