// Small-token (AR decode) path over 4-bit expert weights: T <= 16 tokens, the
// layer a stream over the active experts' codes.
//
//   1. the router partials of decode.hip;
//   2. q4_decode_w13: one workgroup of 16 waves per CU.  It stages the tokens'
//      rows in LDS, runs the routing finish, and streams an equal share of the
//      (active expert, 8 intermediate columns) units: a unit is one row tile
//      of w1 (8 gate rows and their 8 up rows) over all of H, 16 codes tiles of
//      1 KB per 2048 columns, straight to registers in operand order.  Waves
//      take whole units; the units that do not fill all 16 waves (all of them,
//      when few experts are active) are cut along H into 16 equal parts, whose
//      sums are added through LDS in a fixed order.
//   3. q4_decode_down: one workgroup per 16 output columns; its waves take
//      equal parts of the flat list (active expert, micro-shard, 128 columns),
//      matrix rows being the tokens (a token without the expert enters as
//      zeros), so one accumulator gathers w[t, j] * y over all experts of a
//      wave and the 16 waves' sums are the output.
#include "decode_route.h"
#include "q4.h"

namespace moe {
namespace {

constexpr int kDqWaves = 16;
constexpr int kDqBlocks = 256;  // one workgroup per CU
constexpr size_t kDqMaxRows = (size_t)kDecT * 4096 * 2;  // LDS bytes of the staged rows
constexpr int kDqStep = 4;      // code tiles per step: 4 KB a wave in flight, twice

struct Q4DecodeArgs {
  const uint16_t* x;
  const double* partial;
  const float* bias;
  const uint8_t* codes;
  const uint16_t* scales;
  int T, H, E, k, Im, mu, renorm, KB, S;
  uint16_t* h;
  float* logits;
  int32_t* ids;
  float* topw;
  int32_t *counts, *offsets, *perm, *inv, *active;
};

template <int GPB>
struct Step {
  uint4 c[kDqStep];
  float s[kDqStep][GPB];
};

// One 128-column tile: a group's sum on the matrix pipe, then times its scale.
// INT4 operands are 128 + code; a product with -136 everywhere takes the
// excess off again (the matrix pipe idles on this path).
template <int FMT, int GPB, typename F>
__device__ __forceinline__ void tile_mma(const uint4& c, const float (&s)[GPB], F row_operand, f32x4& acc) {
  constexpr int JG = 4 / GPB;
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  const uint4 off = make_uint4(0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u);  // bf16 -136
#pragma unroll
  for (int gr = 0; gr < GPB; ++gr) {
    f32x4 part = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int jj = 0; jj < JG; ++jj) {
      const int j = gr * JG + jj;
      const bf16x8 a = row_operand(j);
      if constexpr (FMT == kQ4Int)
        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, off), part, 0, 0, 0);
      part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, q4_operand<FMT>(w[j]), part, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(s[gr], part[r], acc[r]);
  }
}

template <int FMT, int GPB>
__global__ __launch_bounds__(kDqWaves * 64) void q4_decode_w13(Q4DecodeArgs a) {
  __shared__ RouteLds rs;
  __shared__ __attribute__((aligned(1024))) char xl[kDqMaxRows];  // T rows of H, later the parts' sums
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, g = lane >> 4;

  // the tokens' rows, 16-byte chunks XOR-swizzled by the token
  {
    const int per = a.H / 8;  // chunks of a row (a multiple of 256)
    for (int q = tid; q < a.T * per; q += kDqWaves * 64) {
      const int t = q / per, c = q - t * per;
      *reinterpret_cast<uint4*>(xl + ((size_t)t * per + (c ^ t)) * 16) =
          *reinterpret_cast<const uint4*>(a.x + (size_t)t * a.H + c * 8);
    }
  }
  route_finish(a.partial, a.bias, a.T, a.E, a.k, a.renorm != 0, blockIdx.x == 0, a.logits, a.ids, a.topw, a.counts,
               a.offsets, a.perm, a.inv, a.active, rs);

  const int per_mat = a.Im / 8;                 // units of one matrix
  const int ue = a.mu * per_mat;                // units of one expert
  const int units = rs.act[kMaxExperts] * ue;
  const int u0 = (int)((long long)blockIdx.x * units / gridDim.x);
  const int nu = (int)((long long)(blockIdx.x + 1) * units / gridDim.x) - u0;
  const int full = nu / kDqWaves, rem = nu - full * kDqWaves;
  const int KB = a.KB;
  // this wave's part of the remaining units, in tiles of the flat (unit, tile) list
  const int pa = wave * rem * KB / kDqWaves, pb = (wave + 1) * rem * KB / kDqWaves;
  const int ua = rem > 0 ? pa / KB : 0;
  const int nseg = full + (pb > pa ? 1 + (pb - 1) / KB - ua : 0);

  struct Seg {
    int u, k0, k1;
  };
  auto segment = [&](int i) -> Seg {
    if (i < full) return {u0 + i * kDqWaves + wave, 0, KB};
    const int un = ua + i - full;
    return {u0 + full * kDqWaves + un, max(pa, un * KB) - un * KB, min(pb, (un + 1) * KB) - un * KB};
  };
  const uint8_t* cp = nullptr;   // this lane's codes and scales of the segment being loaded
  const uint16_t* sp = nullptr;
  auto locate = [&](int u) {
    const int e = rs.act[u / ue], r = u % ue;
    const size_t rt = ((size_t)(r / per_mat) * a.E + e) * per_mat + r % per_mat;  // row tile: 2 Im / 16 per matrix
    cp = a.codes + rt * KB * kQ4TileBytes + lane * 16;
    sp = a.scales + (rt * 16 + fr) * a.S;
  };
  auto load = [&](int kb, int k1, Step<GPB>& st) {
#pragma unroll
    for (int i = 0; i < kDqStep; ++i) {
      const int b = min(kb + i, k1 - 1);
      st.c[i] = *reinterpret_cast<const uint4*>(cp + (size_t)b * kQ4TileBytes);
      q4_load_scales<GPB>(sp + b * GPB, st.s[i]);
    }
  };

  f32x4 piece[2];  // sums of this wave's parts
  piece[0] = piece[1] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (nseg > 0) {
    Step<GPB> cur, nxt;
    int si = 0;
    Seg seg = segment(0);
    int kb = seg.k0;
    locate(seg.u);
    load(kb, seg.k1, cur);
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
    while (true) {
      // the next step's loads go out before this one is used
      Seg ns = seg;
      int nk = kb + kDqStep, nsi = si;
      if (nk >= seg.k1) {
        nsi = si + 1;
        if (nsi < nseg) {
          ns = segment(nsi);
          nk = ns.k0;
          locate(ns.u);
        }
      }
      if (nsi < nseg) load(nk, ns.k1, nxt);
      const int e = rs.act[seg.u / ue];
      const int first = rs.off[e], n = rs.off[e + 1] - first;
      // rows past the expert's repeat its last token: never stored
      const int t = rs.perm[first + min(fr, n - 1)] / a.k;
      const char* row = xl + (size_t)t * a.H * 2;
#pragma unroll
      for (int i = 0; i < kDqStep; ++i)
        if (kb + i < seg.k1)
          tile_mma<FMT, GPB>(cur.c[i], cur.s[i],
                             [&](int j) {
                               return *reinterpret_cast<const bf16x8*>(row + ((kb + i) * 16 + ((4 * j + g) ^ t)) * 16);
                             },
                             acc);
      if (nsi != si) {
        if (si < full) {
          // a whole unit: column fr < 8 gate, fr + 8 its up
          const int r8 = seg.u % ue;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float up = __shfl_xor(acc[r], 8);
            const int rowi = 4 * g + r;
            if (fr < 8 && rowi < n)
              a.h[(size_t)(first + rowi) * (a.mu * a.Im) + r8 * 8 + fr] = float_to_bf16_bits(silu_f32(acc[r]) * up);
          }
        } else {
          piece[0] = piece[1];
          piece[1] = acc;
        }
        acc = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      if (nsi >= nseg) break;
      si = nsi;
      seg = ns;
      kb = nk;
      cur = nxt;
    }
  }
  if (rem == 0) return;  // the same for the whole workgroup

  // sums of the cut units: wave w's parts are units ua .. (last first in
  // `piece` order), each part to a slot of its own, then added in wave order
  __syncthreads();
  f32x4* slots = reinterpret_cast<f32x4*>(xl);  // [wave][2][64]
  const int np = nseg - full;
  if (np == 1) slots[(wave * 2 + 0) * 64 + lane] = piece[1];
  if (np == 2) {
    slots[(wave * 2 + 0) * 64 + lane] = piece[0];
    slots[(wave * 2 + 1) * 64 + lane] = piece[1];
  }
  __syncthreads();
  if (wave >= rem) return;
  {
    const int un = wave;  // one wave per cut unit (rem < 16)
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int w = 0; w < kDqWaves; ++w) {
      const int wa = w * rem * KB / kDqWaves, wb = (w + 1) * rem * KB / kDqWaves;
      if (wb <= wa || wb <= un * KB || wa >= (un + 1) * KB) continue;
      const f32x4 v = slots[(w * 2 + (un - wa / KB)) * 64 + lane];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] += v[r];
    }
    const int u = u0 + full * kDqWaves + un;
    const int e = rs.act[u / ue], first = rs.off[e], n = rs.off[e + 1] - first;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float up = __shfl_xor(acc[r], 8);
      const int rowi = 4 * g + r;
      if (fr < 8 && rowi < n)
        a.h[(size_t)(first + rowi) * (a.mu * a.Im) + (u % ue) * 8 + fr] = float_to_bf16_bits(silu_f32(acc[r]) * up);
    }
  }
}

// ---------------------------------------------------------------------------
struct Q4DownArgs {
  const uint16_t* h;
  const int32_t *ids, *inv, *active;
  const float* topw;
  const uint8_t* codes;
  const uint16_t* scales;
  int T, H, E, k, Im, mu, KB, S;
  uint16_t* out;
};

template <int FMT, int GPB>
__global__ __launch_bounds__(kDqWaves * 64) void q4_decode_down(Q4DownArgs a) {
  __shared__ int pos[kMaxExperts][kDecT];     // row of h of (expert, token), or -1
  __shared__ __attribute__((aligned(16))) float wt[kMaxExperts][kDecT];  // its routing weight, or 0
  __shared__ f32x4 part[kDqWaves][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, g = lane >> 4;
  static_assert(kDqWaves * 64 == kMaxExperts * kDecT, "one thread per (expert, token)");
  (&pos[0][0])[tid] = -1;
  (&wt[0][0])[tid] = 0.0f;
  __syncthreads();
  for (int r = tid; r < a.T * a.k; r += kDqWaves * 64) {
    const int e = a.ids[r], t = r / a.k;
    pos[e][t] = a.inv[r];
    wt[e][t] = a.topw[r];
  }
  __syncthreads();

  const int KB = a.KB, per = a.mu * KB;                 // tiles of one expert
  const int total = a.active[kMaxExperts] * per;
  const int q0 = wave * total / kDqWaves, q1 = (wave + 1) * total / kDqWaves;
  const int I = a.mu * a.Im;
  const size_t rt = blockIdx.x;                         // row tile of one matrix
  const size_t mat_tiles = (size_t)a.H / 16;

  auto load = [&](int q, Step<GPB>& st) {
#pragma unroll
    for (int i = 0; i < kDqStep; ++i) {
      const int b = min(q + i, q1 - 1);
      const int ai = b / per, rest = b - ai * per, m = rest / KB, kb = rest - m * KB;
      const size_t tile = ((size_t)m * a.E + a.active[ai]) * mat_tiles + rt;
      st.c[i] = *reinterpret_cast<const uint4*>(a.codes + (tile * KB + kb) * kQ4TileBytes + lane * 16);
      q4_load_scales<GPB>(a.scales + (tile * 16 + fr) * a.S + kb * GPB, st.s[i]);
    }
  };
  f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
  if (q1 > q0) {
    Step<GPB> cur, nxt;
    load(q0, cur);
    for (int q = q0; q < q1; q += kDqStep) {
      if (q + kDqStep < q1) load(q + kDqStep, nxt);
      uint4 av[kDqStep][4];
      int ex[kDqStep];
#pragma unroll
      for (int i = 0; i < kDqStep; ++i) {
        const int b = min(q + i, q1 - 1);
        const int ai = b / per, rest = b - ai * per, m = rest / KB, kb = rest - m * KB;
        const int e = a.active[ai];
        ex[i] = e;
        const int p = pos[e][fr];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = kb * kQ4TileK + 32 * j + 8 * g;
          const bool ok = p >= 0 && c < a.Im;
          const uint4 v = *reinterpret_cast<const uint4*>(a.h + (ok ? (size_t)p * I + m * a.Im + c : 0));
          av[i][j] = ok ? v : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < kDqStep; ++i)
        if (q + i < q1) {
          f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
          tile_mma<FMT, GPB>(cur.c[i], cur.s[i], [&](int j) { return __builtin_bit_cast(bf16x8, av[i][j]); }, acc);
          const f32x4 w = *reinterpret_cast<const f32x4*>(&wt[ex[i]][4 * g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) sum[r] = fmaf(w[r], acc[r], sum[r]);
        }
      cur = nxt;
    }
  }
  part[wave][lane] = sum;
  __syncthreads();
  // D layout: register r of lane (g, fr) holds token 4 g + r, column fr
  if (tid < kDecT * 16) {
    const int t = tid >> 4, c = tid & 15;
    if (t < a.T) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kDqWaves; ++w) s += part[w][(t >> 2) * 16 + c][t & 3];
      a.out[(size_t)t * a.H + blockIdx.x * 16 + c] = float_to_bf16_bits(s);
    }
  }
}

template <int FMT, int GPB>
hipError_t launch_fmt(const Q4DecodeArgs& w, const Q4DownArgs& d, hipStream_t st) {
  hipLaunchKernelGGL((q4_decode_w13<FMT, GPB>), dim3(kDqBlocks), dim3(kDqWaves * 64), 0, st, w);
  hipLaunchKernelGGL((q4_decode_down<FMT, GPB>), dim3(d.H / 16), dim3(kDqWaves * 64), 0, st, d);
  return hipGetLastError();
}

}  // namespace

bool q4_decode_supported(const Shape& s) {
  return s.bf16 && s.T >= 1 && s.T <= kDecT && s.k <= kMaxK && s.H % (kSplit * 128) == 0 &&
         (size_t)s.T * s.H * 2 <= kDqMaxRows;
}

hipError_t launch_q4_decode(const Shape& s, const Q4& q, const void* x, const float* wg, const float* bias,
                            const void* w1c, const void* w1s, const void* w2c, const void* w2s, void* out,
                            float* logits, int32_t* ids, float* w, int32_t* counts, int32_t* offsets, int32_t* perm,
                            int32_t* inv, void* h, void* scratch, hipStream_t st) {
  double* partial = (double*)scratch;
  int32_t* active = (int32_t*)((char*)scratch + kRoutePartialBytes);
  if (const hipError_t e = launch_decode_route_partial(s, x, wg, partial, st); e != hipSuccess) return e;
  const Q4DecodeArgs a = {(const uint16_t*)x, partial, bias, (const uint8_t*)w1c, (const uint16_t*)w1s,
                          s.T, s.H, s.E, s.k, s.Im, s.mu, (int)s.renorm, q.kb(s.H), q.stride(s.H),
                          (uint16_t*)h, logits, ids, w, counts, offsets, perm, inv, active};
  const Q4DownArgs d = {(const uint16_t*)h, ids, inv, active, w, (const uint8_t*)w2c, (const uint16_t*)w2s,
                        s.T, s.H, s.E, s.k, s.Im, s.mu, q.kb(s.Im), q.stride(s.Im), (uint16_t*)out};
  if (q.format == kQ4Int)
    return q.group == 128  ? launch_fmt<kQ4Int, 1>(a, d, st)
           : q.group == 64 ? launch_fmt<kQ4Int, 2>(a, d, st)
                           : launch_fmt<kQ4Int, 4>(a, d, st);
  return q.group == 128  ? launch_fmt<kQ4E2m1, 1>(a, d, st)
         : q.group == 64 ? launch_fmt<kQ4E2m1, 2>(a, d, st)
                         : launch_fmt<kQ4E2m1, 4>(a, d, st);
}

}  // namespace moe
