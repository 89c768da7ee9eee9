// Routing of a small-token batch, shared by the weight-streaming paths
// (decode.hip, q4_decode.hip): the router partials' geometry and the routing
// finish that a workgroup runs for itself.
#pragma once

#include "moe_common.h"

namespace moe {

constexpr int kDecT = 16;       // token tile (max tokens on this path)
constexpr int kSplit = 16;      // router split of the hidden dimension
constexpr int kMaxK = 64;

// Bytes of the router partials; the active-expert list follows them in the
// scratch region of the workspace.
constexpr size_t kRoutePartialBytes = (size_t)kSplit * kDecT * kMaxExperts * sizeof(double);

// fp64 router partial sums of the T <= kDecT tokens (decode.hip).
hipError_t launch_decode_route_partial(const Shape& s, const void* x, const float* wg, double* partial,
                                       hipStream_t st);

// Routing of any number of tokens from such partials, one set per tile of
// kDecT tokens (route_tiles_bytes in all; bf16, H % (kSplit * 128) == 0):
// launch_route's outputs, the logits summed in another order (decode.hip).
size_t route_tiles_bytes(const Shape& s);
hipError_t launch_route_tiles(const Shape& s, const void* x, const float* wg, const float* bias, double* partial,
                              float* logits, int32_t* ids, float* w, int32_t* hist, hipStream_t st);

namespace {

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// ---------------------------------------------------------------------------
// 2. routing of the token tile, run by one workgroup of 16 waves (each
// workgroup of decode_w13 runs it for itself at its start: the inputs are the
// router partials, 128 KB in L2, and the work is a few microseconds, less
// than a separate launch and kernel boundary).  Workgroup `out` writes the
// routing outputs to memory; every workgroup keeps the offsets, the active
// experts and the permutation in LDS for its own use.
struct RouteLds {
  float lg[kDecT][kMaxExperts];
  int sids[kDecT * kMaxK];
  uint64_t sel[kDecT];           // experts chosen by each token
  int base[kMaxExperts];
  int off[kMaxExperts + 1];      // expert offsets
  int act[kMaxExperts + 1];      // active experts ascending; their number in act[kMaxExperts]
  int perm[kDecT * kMaxK];       // permuted row -> route
};

//
// `meanwhile` runs once the partials are summed and before the first barrier:
// work of the caller whose own loads were issued before the call.
template <typename F>
__device__ __forceinline__ void route_finish(
    const double* __restrict__ partial, const float* __restrict__ bias, int T, int E, int k, bool renorm,
    bool out, float* __restrict__ logits, int32_t* __restrict__ ids, float* __restrict__ topw,
    int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ perm,
    int32_t* __restrict__ inv, int32_t* __restrict__ active, RouteLds& S, F meanwhile) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;

  {  // logits: thread (r, e), partials summed in split order (rows past T
     // are never ranked: their partials are not read)
    const int r = tid >> 6, e = tid & 63;
    double s = 0.0;
    if (r < T)
      for (int b = 0; b < kSplit; ++b) s += partial[((size_t)b * kDecT + r) * kMaxExperts + e];
    const double bb = (bias != nullptr && e < E) ? (double)bias[e] : 0.0;
    const float L = (float)(s + bb);
    S.lg[r][e] = L;
    if (out && r < T && e < E) logits[(size_t)r * E + e] = L;
  }
  meanwhile();
  __syncthreads();

  {  // top-k and weights: wave = token, lane = expert (same rules as route.hip)
    const int t = wave;
    if (t < T) {
      uint32_t key = lane < E ? orderable(S.lg[t][lane]) : 0u;
      bool taken = false;
      float mine = 0.0f, first = 0.0f;
      for (int j = 0; j < k; ++j) {
        const uint32_t m = wave_max_u32(key);
        const int win = __ffsll((long long)__ballot(key == m)) - 1;
        const float Lw = from_orderable(m);
        if (j == 0) first = Lw;
        if (lane == j) mine = Lw;
        if (lane == win) {
          key = 0;
          taken = true;
        }
        if (lane == 0) {
          if (out) ids[(size_t)t * k + j] = win;
          S.sids[t * k + j] = win;
        }
      }
      const uint64_t chosen = __ballot(taken);
      if (lane == 0) S.sel[t] = chosen;
      const double ex = (lane < k) ? exp((double)mine - (double)first) : 0.0;
      const double s =
          wave_sum_f64(renorm ? ex : (lane < E ? exp((double)S.lg[t][lane] - (double)first) : 0.0));
      if (out && lane < k) topw[(size_t)t * k + lane] = (float)(ex / s);
    }
  }
  __syncthreads();

  // counts, offsets, active list (wave 0, lane = expert): a token chooses an
  // expert at most once, so the count is the number of tokens whose
  // selection holds it
  const int R = T * k;
  if (wave == 0) {
    int c = 0;
    for (int t = 0; t < T; ++t) c += (int)((S.sel[t] >> lane) & 1ull);
    int incl = c;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    const int excl = incl - c;
    S.base[lane] = excl;
    if (lane < E) {
      S.off[lane] = excl;
      if (out) {
        counts[lane] = c;
        offsets[lane] = excl;
      }
    }
    if (lane == E - 1) {
      S.off[E] = incl;
      if (out) offsets[E] = incl;
    }
    // active experts in ascending order: position = number of active experts below
    const uint64_t act = __ballot(lane < E && c > 0);
    const uint64_t below = (lane == 0) ? 0ull : (act & ((~0ull) >> (64 - lane)));
    if (lane < E && c > 0) {
      S.act[__popcll(below)] = lane;
      if (out) active[__popcll(below)] = lane;
    }
    if (lane == 0) {
      S.act[kMaxExperts] = __popcll(act);
      if (out) active[kMaxExperts] = __popcll(act);
    }
  }
  __syncthreads();
  // stable scatter: the routes of expert e before r = t*k + j are those of
  // the earlier tokens that chose e
  for (int r = tid; r < R; r += blockDim.x) {
    const int t = r / k, e = S.sids[r];
    int rank = 0;
    for (int q = 0; q < t; ++q) rank += (int)((S.sel[q] >> e) & 1ull);
    const int p = S.base[e] + rank;
    S.perm[p] = r;
    if (out) {
      perm[p] = r;
      inv[r] = p;
    }
  }
  __syncthreads();
}

}  // namespace
}  // namespace moe
