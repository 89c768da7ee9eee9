// Small-token (AR decode) path over 4-bit expert weights: T <= 16 tokens, the
// layer a stream over the active experts' codes.
//
//   1. the router partials of decode.hip;
//   2. q4_decode_w13: one workgroup of 16 waves per CU.  It stages the tokens'
//      rows in LDS, runs the routing finish, and streams an equal share of the
//      (active expert, 8 intermediate columns) units: a unit is one row tile
//      of w1 (8 gate rows and their 8 up rows) over all of H, 16 code tiles of
//      1 KB per 2048 columns, straight to registers in operand order.  Matrix
//      rows are the tokens, whatever the expert (rows of tokens that did not
//      choose it are computed and dropped), so a wave's row operands do not
//      depend on its unit.  Waves take whole units; the units that do not fill
//      all 16 waves (all of them, when few experts are active) are cut along H
//      into 16 equal parts, whose sums are added through LDS in a fixed order.
//   3. q4_decode_down: one workgroup per 16 output columns; its waves take
//      equal parts of the flat list (active expert, micro-shard, 128 columns).
//      Matrix rows are again the tokens (one without the expert enters as
//      zeros), so one accumulator gathers w[t, j] * y over all experts of a
//      wave and the 16 waves' sums are the output.
// Bound: the layer H = 4096, E = 64, k = 8, Im = 768 at T = 8 (42 active experts, 198
// MB, INT4, group 128) takes 5 + 35 + 24 us; the codes arrive at about 5.7 TB/s
// once a kernel streams, and each launch, the routing finish, the rows' way to
// LDS and the last sums (about 9 us a kernel) stand before and behind the stream.
// At T = 16 (groups of 32, E2M1: 5 + 54 + 33 us) the rows of h pass LDS in two
// rounds, and the codes of the second are asked for only when its rows are.
// Parts cut in units of four tiles instead of eight: 92 against 92 us at T = 16, 68
// against 64 at T = 8; not kept.
// Both ask for 8 KB of codes a wave ahead (128 KB a CU) and for a tile's
// successor as soon as its registers are free.  In the down product at groups of
// 128 the compiler does not keep that up: it widens the ring's eight 16-bit scales
// together at the end of a pass, behind a wait for every load, so that the ring
// runs empty every eight tiles (and the first time before the staged rows' own
// wait).  At groups of 64 and 32, whose scales come in whole words, it waits for a
// tile's loads alone.  The loads are nontemporal (the
// layer at T = 8: 64.5 against 67.9 us in the kernel trace, at T = 16 with
// groups of 32: 92 against 100 us).
#include "decode_route.h"
#include "q4.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kDqWaves = 16;
constexpr int kDqBlocks = 256;  // one workgroup per CU
constexpr size_t kDqMaxRows = (size_t)kDecT * 4096 * 2;  // LDS bytes of the staged rows
constexpr int kDqRing = 8;  // code tiles a wave keeps in flight: 8 KB

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

// Scales stay as loaded (bf16, two a word): a conversion would wait for the
// loads where they are issued.  (A single one, load_tile_scales<1>, is widened to
// its word there: see the top.)
// The scales of four neighbouring tiles (8 GPB bytes, aligned to that).
template <int GPB>
__device__ __forceinline__ void load_step_scales(const uint16_t* p, uint32_t (&s)[2 * GPB]) {
  if constexpr (GPB == 1) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    s[0] = v.x;
    s[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < GPB / 2; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      s[4 * i] = v.x;
      s[4 * i + 1] = v.y;
      s[4 * i + 2] = v.z;
      s[4 * i + 3] = v.w;
    }
  }
}
// The scales of one tile.
template <int GPB>
__device__ __forceinline__ void load_tile_scales(const uint16_t* p, uint32_t (&s)[(GPB + 1) / 2]) {
  if constexpr (GPB == 1) {
    s[0] = *p;
  } else if constexpr (GPB == 2) {
    s[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    s[0] = v.x;
    s[1] = v.y;
  }
}
__device__ __forceinline__ float half_scale(uint32_t w, int i) {
  return __uint_as_float((i & 1) ? w & 0xffff0000u : w << 16);
}

// One 128-column tile: a group's sum on the matrix pipe, from start(group) on,
// then times its scale.  INT4 operands are 128 + code: their sums start at
// -136 times the rows' sums over the group.
template <int FMT, int GPB, typename F, typename G>
__device__ __forceinline__ void tile_mma(const uint4& c, const float (&s)[GPB], const Q4Consts& kc, F row_operand,
                                         G start, f32x4& acc) {
  constexpr int JG = 4 / GPB;
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int gr = 0; gr < GPB; ++gr) {
    f32x4 part = FMT == kQ4Int ? start(gr) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = gr * JG; j < (gr + 1) * JG; ++j)
      part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(row_operand(j), q4_operand<FMT>(w[j], kc), part, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(s[gr], part[r], acc[r]);
  }
  pin(acc);
}

constexpr int kDqStage = (int)(kDqMaxRows / 16 / (kDqWaves * 64));  // 16-byte chunks a thread stages, at most
constexpr int kDqSums = kDecT * 4096 / 32;                          // sums of row groups, at most

template <int FMT, int GPB>
__global__ __launch_bounds__(kDqWaves * 64) void q4_decode_w13(Q4DecodeArgs a) {
  __shared__ RouteLds rs;
  __shared__ __attribute__((aligned(8))) short pos[kMaxExperts][kDecT];  // row of h of (expert, token), or -1
  __shared__ __attribute__((aligned(16))) float xsum[FMT == kQ4Int ? kDqSums : 4];  // [group][token], times -136
  __shared__ __attribute__((aligned(1024))) char xl[kDqMaxRows];  // T rows of H, later the parts' sums
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, g = lane >> 4;
  const int Tp = (a.T + 3) & ~3;                // tokens of a row of xsum
  const int chunks = a.T * (a.H / 8);           // 16-byte chunks of the tokens' rows

  // the rows are on their way while the routing's partial sums are read (INT4; in
  // the E2M1 instances the compiler keeps xv in private memory, 144 bytes a lane,
  // and waits for one chunk before it asks for the next: up to eight round
  // trips at T = 16); then to LDS, chunks XOR-swizzled by the token, and their groups' sums.  64
  // neighbouring chunks are one token's (H / 8 is a multiple of 256).
  uint4 xv[kDqStage];
#pragma unroll
  for (int i = 0; i < kDqStage; ++i) {
    const int q0 = (i * kDqWaves + wave) * 64;
    if (q0 < chunks) xv[i] = reinterpret_cast<const uint4*>(a.x)[q0 + lane];
  }
  (&pos[0][0])[tid] = -1;
  auto stage = [&] {
#pragma unroll
    for (int i = 0; i < kDqStage; ++i) {
      const int q0 = (i * kDqWaves + wave) * 64;
      if (q0 < chunks) {
        const int t = q0 / (a.H / 8), c = q0 - t * (a.H / 8) + lane;
        *reinterpret_cast<uint4*>(xl + (t * (a.H / 8) + (c ^ t)) * 16) = xv[i];
        if constexpr (FMT == kQ4Int) {
          const float sum = q4_group_start<GPB>(xv[i]);
          if ((lane & (16 / GPB - 1)) == 0) xsum[c / (16 / GPB) * Tp + t] = sum;
        }
      }
    }
  };
  route_finish(a.partial, a.bias, a.T, a.E, a.k, a.renorm != 0, blockIdx.x == 0, a.logits, a.ids, a.topw, a.counts,
               a.offsets, a.perm, a.inv, a.active, rs, stage);
  static_assert(kDqWaves * 64 == kMaxExperts * kDecT && kDecT * kMaxK <= kDqWaves * 64, "one thread per entry and route");
  if (tid < a.T * a.k) {
    const int r = rs.perm[tid];
    pos[rs.sids[r]][r / a.k] = (short)tid;
  }

  const int per_mat = a.Im / 8;                 // units of one matrix
  const int ue = a.mu * per_mat;                // units of one expert
  const int units = rs.act[kMaxExperts] * ue;
  const int u0 = (int)((long long)blockIdx.x * units / gridDim.x);
  const int nu = (int)((long long)(blockIdx.x + 1) * units / gridDim.x) - u0;
  const int full = nu / kDqWaves, rem = nu - full * kDqWaves;
  const int KB = a.KB;
  // this wave's part of the remaining units, in whole rings of the flat (unit, tile) list (KB % 16 == 0)
  auto part_at = [&](int w) { return w * rem * (KB / kDqRing) / kDqWaves * kDqRing; };
  const int pa = part_at(wave), pb = part_at(wave + 1);
  const int ua = rem > 0 ? pa / KB : 0;
  const int nseg = full + (pb > pa ? 1 + (pb - 1) / KB - ua : 0);

  // segment i of this wave: a unit, its end tile, and where its weights and results lie
  struct Seg {
    int k1, e, col;          // end tile, expert, first column of h
    const uint8_t* cp;       // this lane's codes and scales
    const uint16_t* sp;
  };
  int k_first = 0;           // first tile of the segment last asked for
  auto segment = [&](int i) -> Seg {
    int u, k1 = KB;
    k_first = 0;
    if (i < full) {
      u = u0 + i * kDqWaves + wave;
    } else {
      const int un = ua + i - full;
      u = u0 + full * kDqWaves + un;
      k_first = max(pa, un * KB) - un * KB;
      k1 = min(pb, (un + 1) * KB) - un * KB;
    }
    const int ai = u / ue, r = u - ai * ue, m = r / per_mat;
    const int e = __builtin_amdgcn_readfirstlane(rs.act[ai]);
    const size_t rt = ((size_t)m * a.E + e) * per_mat + (r - m * per_mat);  // row tile: 2 Im / 16 per matrix
    return {k1, e, r * 8, a.codes + rt * KB * kQ4TileBytes + lane * 16, a.scales + (rt * 16 + fr) * a.S};
  };
  uint4 ring[kDqRing];
  uint32_t rsc[kDqRing / 4][2 * GPB];
  auto load_tile = [&](const Seg& sg, int kb, int i) {
    ring[i] = load_codes<true>(sg.cp + (size_t)(kb + i) * kQ4TileBytes);
    if ((i & 3) == 3) load_step_scales<GPB>(sg.sp + (kb + i - 3) * GPB, rsc[i / 4]);
  };
  auto store_h = [&](int e, int col, const f32x4& v) {
    // tile columns 0-7 gate, 8-15 the up columns of the same 8.  h is rounded to the
    // layer's type, as the step-wise products and the dense layer do: it is an output
    // of the workspace, and the down product's operands are bf16.  (With h and y in
    // fp32 the output would be 0.0017 from the 64-bit result instead of 0.0024.)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float up = __shfl_xor(v[r], 8);
      const int p = pos[e][4 * g + r];
      if (fr < 8 && p >= 0)
        a.h[(size_t)p * (a.mu * a.Im) + col + fr] = float_to_bf16_bits(silu_f32(v[r]) * up);
    }
  };

  const Q4Consts kc;
  Seg seg = {0, 0, 0, nullptr, nullptr};
  int kb = 0;
  if (nseg > 0) {
    seg = segment(0);
    kb = k_first;
#pragma unroll
    for (int i = 0; i < kDqRing; ++i) load_tile(seg, kb, i);
  }
  __builtin_amdgcn_sched_barrier(0);
  lds_barrier();  // pos is written

  f32x4 piece[2];  // sums of this wave's parts
  piece[0] = piece[1] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (nseg > 0) {
    int si = 0;
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
    // this lane's row operand: token fr (tokens past the last repeat it: never stored)
    const uint32_t t = min(fr, a.T - 1);
    uint32_t row[4];  // LDS offsets of its chunks of tile 0
#pragma unroll
    for (int j = 0; j < 4; ++j) row[j] = t * (uint32_t)a.H * 2u + (((4u * j + g) ^ t) * 16u);
    const float* sums = xsum + 4 * min(g, Tp / 4 - 1);  // tokens 4 g .. 4 g + 3
    // the products of the ring's 8 tiles from tile kb on, each tile's registers refilled with one of the next 8
    auto products = [&](auto refill, const Seg& ns, int nk) {
      const char* base = xl + kb * (kQ4TileK * 2);
#pragma unroll
      for (int i = 0; i < kDqRing; ++i) {
        float sc[GPB];
#pragma unroll
        for (int q = 0; q < GPB; ++q) sc[q] = half_scale(rsc[i / 4][((i & 3) * GPB + q) >> 1], (i & 3) * GPB + q);
        tile_mma<FMT, GPB>(
            ring[i], sc, kc,
            [&](int j) { return *reinterpret_cast<const bf16x8*>(base + row[j] + i * (kQ4TileK * 2)); },
            [&](int gr) { return *reinterpret_cast<const f32x4*>(sums + ((kb + i) * GPB + gr) * Tp); }, acc);
        if constexpr (decltype(refill)::value) load_tile(ns, nk, i);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto finish = [&]() {  // the sums of this wave's share of the segment are complete
      if (si < full) {
        store_h(seg.e, seg.col, acc);
      } else {
        piece[0] = piece[1];
        piece[1] = acc;
      }
      acc = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    while (true) {
      const bool same = kb + kDqRing < seg.k1;
      if (!same && si + 1 >= nseg) break;
      Seg ns = seg;
      int nk = kb + kDqRing;
      if (!same) {
        ns = segment(si + 1);
        nk = k_first;
      }
      products(std::true_type{}, ns, nk);
      kb = nk;
      if (!same) {
        finish();
        ++si;
        seg = ns;
      }
    }
    products(std::false_type{}, seg, 0);
    finish();
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
      const int wa = part_at(w), wb = part_at(w + 1);
      if (wb <= wa || wb <= un * KB || wa >= (un + 1) * KB) continue;
      const f32x4 v = slots[(w * 2 + (un - wa / KB)) * 64 + lane];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] += v[r];
    }
    const int u = u0 + full * kDqWaves + un, ai = u / ue;
    store_h(rs.act[ai], (u - ai * ue) * 8, acc);
  }
}

// ---------------------------------------------------------------------------
struct Q4DownArgs {
  const uint16_t* h;
  const int32_t *ids, *inv, *offsets, *active;
  const float* topw;
  const uint8_t* codes;
  const uint16_t* scales;
  int T, H, E, k, Im, mu, KB, S;
  uint16_t* out;
};

template <int FMT, int GPB>
__global__ __launch_bounds__(kDqWaves * 64) void q4_decode_down(Q4DownArgs a) {
  // rows of h, 16-byte chunks XOR-swizzled by the row; what a last
  // copy of 64 chunks may add, and 256 zero bytes, the operand of a token without a row
  __shared__ __attribute__((aligned(1024))) char hl[kDqMaxRows + 1024];
  __shared__ short pos[kMaxExperts][kDecT];  // row of h of (expert, token), or -1
  __shared__ __attribute__((aligned(16))) float wt[kMaxExperts][kDecT];  // its routing weight, or 0
  __shared__ int act[kMaxExperts], off[kMaxExperts + 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, g = lane >> 4;
  static_assert(kDqWaves * 64 == kMaxExperts * kDecT, "one thread per (expert, token)");
  (&pos[0][0])[tid] = -1;
  (&wt[0][0])[tid] = 0.0f;
  if (tid < 64) reinterpret_cast<uint32_t*>(hl + kDqMaxRows + 768)[tid] = 0u;
  const int n_act = a.active[kMaxExperts];
  if (tid < kMaxExperts) act[tid] = a.active[tid];  // past n_act: never used
  if (tid <= a.E) off[tid] = a.offsets[tid];
  static_assert(kDqWaves * 64 >= kDecT * kMaxK, "one thread per route");
  const int R = a.T * a.k, rr = min(tid, R - 1);
  const int re = a.ids[rr], rp = a.inv[rr];
  const float rw = a.topw[rr];
  __syncthreads();
  if (tid < R) {
    pos[re][tid / a.k] = (short)rp;
    wt[re][tid / a.k] = rw;
  }

  const int KB = a.KB, per = a.mu * KB;  // tiles of one expert
  const int I = a.mu * a.Im, row_bytes = per * kQ4TileK * 2;
  const int fit = (int)(kDqMaxRows / row_bytes);         // rows that LDS holds, at least T
  const size_t mat_bytes = (size_t)(a.H / 16) * KB * kQ4TileBytes, mat_scales = (size_t)a.H * a.S;
  f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};

  // rounds of as many experts as LDS holds the rows of (one, mostly)
  const Q4Consts kc;
  for (int a0 = 0; a0 < n_act;) {
    const int p0 = off[act[a0]];
    int a1 = a0 + 1;
    while (a1 < n_act && off[act[a1] + 1] - p0 <= fit) ++a1;
    const int q0r = a0 * per, nq = (a1 - a0) * per;
    const int q0 = __builtin_amdgcn_readfirstlane(q0r + wave * nq / kDqWaves);
    const int q1 = __builtin_amdgcn_readfirstlane(q0r + (wave + 1) * nq / kDqWaves);

    // the tile to load next, as its place in the flat list (active expert,
    // micro-shard, tile) and its address; past the wave's last tile the last
    // one is loaded again, and not used
    const int ls = min(q0, q0r + nq - 1);
    int lq = ls, lai = ls / per, lm = (ls - lai * per) / KB, lkb = ls - lai * per - lm * KB;
    const uint8_t* lc;
    const uint16_t* lsc;
    auto matrix = [&]() {
      const size_t mat = (size_t)lm * a.E + __builtin_amdgcn_readfirstlane(act[lai]);
      lc = a.codes + mat * mat_bytes + (size_t)blockIdx.x * KB * kQ4TileBytes + lane * 16;
      lsc = a.scales + mat * mat_scales + ((size_t)blockIdx.x * 16 + fr) * a.S;
    };
    matrix();
    uint4 ring[kDqRing];
    uint32_t rsc[kDqRing][(GPB + 1) / 2];
    auto load_tile = [&](int i) {
      ring[i] = load_codes<true>(lc + (size_t)lkb * kQ4TileBytes);
      load_tile_scales<GPB>(lsc + lkb * GPB, rsc[i]);
      if (lq + 1 < q1) {
        ++lq;
        if (++lkb == KB) {
          lkb = 0;
          if (++lm == a.mu) {
            lm = 0;
            ++lai;
          }
          matrix();
        }
      }
    };
    // rows of the round's experts straight to LDS, each micro-shard's columns
    // padded to whole tiles (the padding meets scales of zero and holds the
    // row's first values); asked for before the codes, and waited for alone
    const int rchunks = row_bytes / 16, staged = (off[act[a1 - 1] + 1] - p0) * rchunks, mc = KB * (kQ4TileK / 8);
    const uint16_t* hbase = uniform_ptr(a.h + (size_t)p0 * I);
    for (int q0s = wave * 64; q0s < staged; q0s += kDqWaves * 64) {
      const int q = min(q0s + lane, staged - 1);  // a row is a multiple of 16 chunks, a wave may end inside the last
      const int r = q / rchunks, c = (q - r * rchunks) ^ ((p0 + r) & 15), m = c / mc, k = (c - m * mc) * 8;
      dma16((uint32_t)(uintptr_t)hl + (uint32_t)q0s * 16u, hbase, (uint32_t)(r * I + m * a.Im + (k < a.Im ? k : 0)) * 2u);
    }
    if (q1 > q0) {
#pragma unroll
      for (int i = 0; i < kDqRing; ++i) load_tile(i);
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<2 * kDqRing>();  // all but the ring's codes and scales
    } else {
      wait_vmcnt<0>();
    }
    lds_barrier();
    if (q1 > q0) {
      int q = q0, cai = q0 / per, ct = q0 - cai * per;  // the tile to compute: active expert, tile of it
      const char* row = nullptr;  // this lane's row of h, or the zeros
      int sw = 0, live = 0;
      f32x4 w = f32x4{0.f, 0.f, 0.f, 0.f}, acc = f32x4{0.f, 0.f, 0.f, 0.f};
      auto enter = [&]() {
        const int e = __builtin_amdgcn_readfirstlane(act[cai]);
        const int p = pos[e][fr];
        row = hl + (p >= 0 ? (p - p0) * row_bytes : (int)kDqMaxRows + 768);
        live = p >= 0 ? ~0 : 0;
        sw = p & 15;
        w = *reinterpret_cast<const f32x4*>(&wt[e][4 * g]);
      };
      auto leave = [&]() {  // the expert's sum of this wave's tiles, times the routing weights
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] = fmaf(w[r], acc[r], sum[r]);
        acc = f32x4{0.f, 0.f, 0.f, 0.f};
      };
      auto products = [&](auto refill) {
#pragma unroll
        for (int i = 0; i < kDqRing; ++i) {
          if (q + i < q1) {
            float sc[GPB];
#pragma unroll
            for (int u = 0; u < GPB; ++u) sc[u] = half_scale(rsc[i][u >> 1], u);
            const char* at = row + ((ct * (kQ4TileK * 2)) & live);
            auto operand = [&](int j) { return *reinterpret_cast<const bf16x8*>(at + (((4 * j + g) ^ sw) * 16)); };
            tile_mma<FMT, GPB>(
                ring[i], sc, kc, operand,
                [&](int gr) {
                  // the rows differ from expert to expert and are used by few tiles: their sums, times -136, by
                  // the matrix pipe itself
                  f32x4 z = f32x4{0.f, 0.f, 0.f, 0.f};
                  const uint4 off136 = make_uint4(0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u);  // bf16 -136
#pragma unroll
                  for (int j = gr * (4 / GPB); j < (gr + 1) * (4 / GPB); ++j)
                    z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(j), __builtin_bit_cast(bf16x8, off136), z, 0, 0, 0);
                  return z;
                },
                acc);
            if (++ct == per) {
              ct = 0;
              ++cai;
              leave();
              if (q + i + 1 < q1) enter();
            }
          }
          if constexpr (decltype(refill)::value) load_tile(i);
          __builtin_amdgcn_sched_barrier(0);
        }
        q += kDqRing;
      };
      enter();
      while (q + kDqRing < q1) products(std::true_type{});
      products(std::false_type{});
      leave();
    }
    __syncthreads();  // the rows are read: the next round's, or the sums, take their place
    a0 = a1;
  }
  f32x4(*part)[64] = reinterpret_cast<f32x4(*)[64]>(hl);
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
         (size_t)((s.T + 3) / 4 * 4) * s.H * 2 <= kDqMaxRows && (size_t)s.T * (s.mu * ((s.Im + 127) / 128) * 256) <= kDqMaxRows;
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
  const Q4DownArgs d = {(const uint16_t*)h, ids, inv, offsets, active, w, (const uint8_t*)w2c, (const uint16_t*)w2s,
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
