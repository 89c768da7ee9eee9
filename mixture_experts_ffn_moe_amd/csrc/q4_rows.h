// Grouped products over 4-bit weights: one template for the gate|up product
// with SwiGLU and for the down product.
//
// A workgroup of 8 waves takes up to 64 rows of one expert (16 MT, MT the
// fewest 16-row tiles that hold them) and 256 weight rows, a wave 32 of them.
// The codes are the bulk of the bytes and each is used once per row block, so
// they go from HBM straight to registers in operand order (a wave loads whole
// 1 KB tiles, 16 bytes a lane), `depth` steps ahead of their use.  The rows'
// operands (x gathered through perm, or h) are shared by the waves: loaded
// equally far ahead, they pass through LDS, double-buffered, one barrier a
// step.  (Loads return in order: were the rows asked for later than the codes,
// waiting for them would wait for every code in flight.)  A row of 256 bytes
// (128 columns) keeps its 16-byte chunks XOR-swizzled by the row, so the 16
// rows of a fragment read hit 16 bank groups.
//
// INT4 codes enter as 128 + code (q4.h).  The 136 * sum(x) too much of a
// group is the same for every weight row, so the thread that stages a chunk
// sums it (8 values, then over the group's lanes), and -136 times the sum
// starts the group's accumulator: no extra matrix instruction.
#pragma once

#include "q4.h"

namespace moe {

struct Q4Rows {
  const void* x;            // rows of operands: x [T, K] through perm, or h [R, segments * K]
  const int32_t* perm;      // w13 only
  const int32_t* offsets;   // [E + 1]
  const uint8_t* codes;
  const void* scales;
  void* out;                // h, or y's values
  int8_t* ye;               // y's exponents (bf16 layers)
  int E, k, K, ldx;         // K: columns of one matrix
  int N;                    // rows of one matrix
  int S;                    // scales per row
  int KB;                   // code tiles along K
  int segments;             // matrices summed into one output (down: micro-shards)
  int tiles;                // output tiles of one expert, all of them (w13: over the micro-shards)
  int Im;                   // w13 only
};

constexpr int kQrWaves = 8;

namespace {

// A row block of an expert: expert, first row and end of the expert's rows.
struct RowBlock {
  int e, row0, end;
};

// The i-th block of MR rows over all experts (blocks of one expert are
// neighbours); e < 0 past the last.  Every wave finds it by itself, one lane
// per expert.
template <int MR>
__device__ __forceinline__ RowBlock find_block(const int32_t* __restrict__ offsets, int E, int i) {
  const int lane = threadIdx.x & 63;
  const int b = offsets[min(lane, E)], n = offsets[min(lane + 1, E)];
  const int blocks = lane < E ? (n - b + MR - 1) / MR : 0;
  int incl = blocks;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  const uint64_t hit = __ballot(i < incl);
  if (hit == 0) return {-1, 0, 0};
  const int e = __ffsll((long long)hit) - 1;
  const int first = __shfl(incl - blocks, e);
  return {e, __shfl(b, e) + (i - first) * MR, __shfl(n, e)};
}

}  // namespace

constexpr int kQrTiles = 2;         // weight row tiles of a wave
constexpr int kQrColTiles = kQrWaves * kQrTiles;
constexpr int kQrLds = 16384;       // bytes of one buffer of staged rows, at most

// An LDS barrier that leaves loads in flight.
__device__ __forceinline__ void q4_lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Keeps the additions that produce v in this block: sunk past a branch, right
// behind the matrix instruction whose result they read, they have been left
// without the wait states that this instruction needs.
__device__ __forceinline__ void q4_pin(f32x4& v) { asm volatile("" : "+v"(v)); }

template <typename XT, int FMT, int GPB, int MT, bool W13>
struct RowsBody {
  static constexpr bool kBf16 = sizeof(XT) == 2;
  static constexpr int NT = kQrTiles;
  static constexpr int MR = 16 * MT;
  static constexpr int KC = MT == 1 ? 2 : 1;           // code tiles per step and weight row tile
  static constexpr int D = !kBf16 ? 2 : MT <= 2 ? 4 : GPB < 4 ? 3 : 2;  // steps in flight (registers allow no more)
  static constexpr int kRowBytes = kQ4TileK * (int)sizeof(XT);
  static constexpr int kChunks = kRowBytes / 16;       // 16-byte chunks of a row's tile
  static constexpr int kStage = KC * MR * kChunks;     // chunks of a step
  static constexpr int kLoads = (kStage + kQrWaves * 64 - 1) / (kQrWaves * 64);
  static constexpr bool kSums = kBf16 && FMT == kQ4Int;
  static constexpr int JG = 4 / GPB;                   // 32-column pieces per group
  static constexpr int SW = kBf16 ? (GPB + 1) / 2 : GPB;  // words of a tile's scales
  static_assert(kStage * 16 <= kQrLds, "a step fits its buffer");

  const Q4Rows& a;
  const RowBlock& blk;
  char* abuf;     // two buffers of kQrLds bytes
  float* xsum;    // two of KC * GPB * MR
  const int tid, lane, wave, fr, g, nb, tile0;
  const Q4Consts kc;

  const uint8_t* codes[NT];
  const XT* scales[NT];
  size_t seg_codes, seg_scales;
  const XT* src[kLoads];
  bool row_ok[kLoads];
  uint4 av[D][kLoads];
  uint4 cw[D][KC][NT];
  uint32_t sw[D][KC][NT][SW];
  f32x4 acc[MT][NT];

  __device__ __forceinline__ RowsBody(const Q4Rows& a_, const RowBlock& b_, int col_wg, char* abuf_, float* xsum_)
      : a(a_), blk(b_), abuf(abuf_), xsum(xsum_), tid(threadIdx.x), lane(threadIdx.x & 63),
        wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), fr(threadIdx.x & 15), g((threadIdx.x & 63) >> 4),
        nb(a_.segments * a_.KB), tile0((col_wg * kQrWaves + wave) * NT) {
    // this wave's output tiles; past the last they repeat it and store nothing
    seg_codes = (size_t)a.E * (a.N / 16) * a.KB * kQ4TileBytes;
    seg_scales = (size_t)a.E * a.N * a.S;
    const int per = a.N / 16;  // row tiles of one matrix
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int ct = min(tile0 + n, a.tiles - 1);
      const int m = W13 ? ct / per : 0, it = W13 ? ct % per : ct;
      const size_t tile = ((size_t)m * a.E + blk.e) * per + it;
      codes[n] = a.codes + tile * a.KB * kQ4TileBytes + lane * 16;
      scales[n] = (const XT*)a.scales + (tile * 16 + fr) * a.S;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int p = blk.row0 + chunk_row(i);
      row_ok[i] = p < blk.end && in_stage(i);
      const int pc = min(p, blk.end - 1);
      src[i] = (const XT*)a.x + (size_t)(W13 ? a.perm[pc] / a.k : pc) * a.ldx;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // chunk i of this thread within a step: tile of the step, row, chunk of the row
  __device__ __forceinline__ int chunk_index(int i) const { return tid + i * kQrWaves * 64; }
  __device__ __forceinline__ bool in_stage(int i) const { return chunk_index(i) < kStage; }
  __device__ __forceinline__ int chunk_col(int i) const { return chunk_index(i) % kChunks; }
  __device__ __forceinline__ int chunk_row(int i) const { return chunk_index(i) / kChunks % MR; }
  __device__ __forceinline__ int chunk_tile(int i) const { return chunk_index(i) / (kChunks * MR); }

  __device__ __forceinline__ void load_rows(int b0, uint4 (&v)[kLoads]) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int b = b0 + chunk_tile(i);
      const int seg = W13 ? 0 : b / a.KB;
      const int col0 = (b - seg * a.KB) * kQ4TileK + chunk_col(i) * (16 / (int)sizeof(XT));  // within the matrix
      const bool ok = row_ok[i] && b < nb && col0 < a.K;
      // a chunk that is not ok loads the row's first columns; it is dropped when it is stored
      v[i] = *reinterpret_cast<const uint4*>(src[i] + (ok ? (size_t)seg * a.K + col0 : 0));
    }
  }
  __device__ __forceinline__ void load_codes(int b0, uint4 (&c)[KC][NT], uint32_t (&s)[KC][NT][SW]) const {
#pragma unroll
    for (int u = 0; u < KC; ++u) {
      const int b = min(b0 + u, nb - 1);  // past the end: loaded again, not used
      const int seg = W13 ? 0 : b / a.KB;
      const int kb = b - seg * a.KB;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        c[u][n] = *reinterpret_cast<const uint4*>(codes[n] + seg * seg_codes + (size_t)kb * kQ4TileBytes);
        const XT* p = scales[n] + seg * seg_scales + kb * GPB;
        if constexpr (!kBf16) {
#pragma unroll
          for (int q = 0; q < GPB; ++q) s[u][n][q] = __float_as_uint(p[q]);
        } else if constexpr (GPB == 1) {
          s[u][n][0] = *p;
        } else {
#pragma unroll
          for (int q = 0; q < SW; ++q) s[u][n][q] = reinterpret_cast<const uint32_t*>(p)[q];
        }
      }
    }
  }
  __device__ __forceinline__ void store_rows(int b0, const uint4 (&v)[kLoads], int buf) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int u = chunk_tile(i), r = chunk_row(i), c = chunk_col(i), b = b0 + u;
      const int kb = W13 ? b : b % a.KB;
      const bool ok = row_ok[i] && b < nb && kb * kQ4TileK + c * (16 / (int)sizeof(XT)) < a.K;
      const uint4 w = ok ? v[i] : make_uint4(0, 0, 0, 0);
      const int x = kBf16 ? (r & 15) : (r & 15) << 1;
      if (in_stage(i))
        *reinterpret_cast<uint4*>(abuf + buf * kQrLds + (u * MR + r) * kRowBytes + ((c ^ x) * 16)) = w;
      if constexpr (kSums) {
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) s += __uint_as_float(q[j] << 16) + __uint_as_float(q[j] & 0xffff0000u);
#pragma unroll
        for (int d = 1; d < kChunks / GPB; d <<= 1) s += __shfl_xor(s, d);
        if ((tid & (kChunks / GPB - 1)) == 0 && in_stage(i))
          xsum[buf * (KC * GPB * MR) + (u * GPB + c / (kChunks / GPB)) * MR + r] = -136.0f * s;
      }
    }
  }
  __device__ __forceinline__ float scale(const uint32_t (&s)[SW], int q) const {
    if constexpr (!kBf16) return __uint_as_float(s[q]);
    return __uint_as_float((q & 1) ? s[q / 2] & 0xffff0000u : s[q / 2] << 16);
  }
  __device__ __forceinline__ void products(int b0, const uint4 (&c)[KC][NT], const uint32_t (&s)[KC][NT][SW], int buf) {
#pragma unroll
    for (int u = 0; u < KC; ++u) {
      if (b0 + u < nb) {
#pragma unroll
        for (int gr = 0; gr < GPB; ++gr) {
          f32x4 part[MT][NT];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            f32x4 start = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (kSums)
              start = *reinterpret_cast<const f32x4*>(&xsum[buf * (KC * GPB * MR) + (u * GPB + gr) * MR + 16 * m + 4 * g]);
#pragma unroll
            for (int n = 0; n < NT; ++n) part[m][n] = start;
          }
#pragma unroll
          for (int j = gr * JG; j < (gr + 1) * JG; ++j) {
            bf16x8 bv[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
              bv[n] = q4_operand<FMT>(j == 0 ? c[u][n].x : j == 1 ? c[u][n].y : j == 2 ? c[u][n].z : c[u][n].w, kc);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const char* row = abuf + buf * kQrLds + (u * MR + 16 * m + fr) * kRowBytes;
              if constexpr (kBf16) {
                const bf16x8 av8 = *reinterpret_cast<const bf16x8*>(row + (((4 * j + g) ^ fr) * 16));
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  part[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av8, bv[n], part[m][n], 0, 0, 0);
              } else {
                // fp32 operands: element i of the four lane groups is one k-step of 4
                const int ch = 2 * (4 * j + g);
                const f32x4 lo = *reinterpret_cast<const f32x4*>(row + ((ch ^ (fr << 1)) * 16));
                const f32x4 hi = *reinterpret_cast<const f32x4*>(row + (((ch + 1) ^ (fr << 1)) * 16));
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                  for (int n = 0; n < NT; ++n)
                    part[m][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(i < 4 ? lo[i] : hi[i - 4], q4_value<FMT>(bv[n], i),
                                                                      part[m][n], 0, 0, 0);
              }
            }
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float f = scale(s[u][n], gr);
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[m][n][r] = fmaf(f, part[m][n][r], acc[m][n][r]);
            }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) q4_pin(acc[m][n]);
  }

  // Step k of the slot d = k mod D: its products, then the slot's codes and the
  // next slot's rows (which go to LDS first) for D steps later.
  template <int d, bool kLoad>
  __device__ __forceinline__ void step(int k) {
    constexpr int e = (d + 1) % D;
    products(k * KC, cw[d], sw[d], k & 1);
    if (kLoad) load_codes((k + D) * KC, cw[d], sw[d]);
    store_rows((k + 1) * KC, av[e], (k + 1) & 1);
    if (kLoad) load_rows((k + 1 + D) * KC, av[e]);
    __builtin_amdgcn_sched_barrier(0);
    q4_lds_barrier();
  }
  template <int d>
  __device__ __forceinline__ void round(int k) {  // D steps with their loads
    if constexpr (d < D) {
      step<d, true>(k + d);
      round<d + 1>(k);
    }
  }
  template <int d>
  __device__ __forceinline__ void last(int k, int steps) {  // up to 2 D - 1 steps; loads only for those there are
    if constexpr (d < 2 * D - 1) {
      if (k + d >= steps) return;
      if (k + d + D < steps)
        step<d % D, true>(k + d);
      else
        step<d % D, false>(k + d);
      last<d + 1>(k, steps);
    }
  }
  template <int d>
  __device__ __forceinline__ void fill() {
    if constexpr (d < D) {
      load_rows(d * KC, av[d]);
      load_codes(d * KC, cw[d], sw[d]);
      fill<d + 1>();
    }
  }
  __device__ __forceinline__ void sums() {
    const int steps = (nb + KC - 1) / KC;
    fill<0>();
    __builtin_amdgcn_sched_barrier(0);
    store_rows(0, av[0], 0);
    load_rows(D * KC, av[0]);
    q4_lds_barrier();
    int k = 0;
    for (; k + 2 * D <= steps; k += D) round<0>(k);
    last<0>(k, steps);
  }

  // D layout of the matrix instruction: register r of a lane holds row 4 (lane/16) + r, column lane%16
  __device__ __forceinline__ int row_of(int m, int r) const { return blk.row0 + 16 * m + 4 * g + r; }

  __device__ __forceinline__ void store_h() const {
    // tile columns 0-7 gate, 8-15 the up columns of the same 8
    const int per = a.N / 16;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int ct = tile0 + n;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float up = __shfl_xor(acc[m][n][r], 8);
          const int p = row_of(m, r);
          if (ct < a.tiles && fr < 8 && p < blk.end)
            ((XT*)a.out)[(size_t)p * (a.tiles * 8) + (ct / per) * a.Im + (ct % per) * 8 + fr] =
                Elem<XT>::from_f(silu_f32(acc[m][n][r]) * up);
        }
    }
  }
  __device__ __forceinline__ void store_y(int col_wg) const {
    if constexpr (!kBf16) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int p = row_of(m, r);
            if (tile0 + n < a.tiles && p < blk.end)
              ((float*)a.out)[(size_t)p * a.N + (tile0 + n) * 16 + fr] = acc[m][n][r];
          }
    } else {
      // block-scaled half y: the workgroup's columns are one block of 256
      // (repeated tiles past H repeat a stored column: the maximum is unchanged)
      static_assert(kQrColTiles * 16 == kYBlock, "one y block per workgroup");
      float* rowmax = reinterpret_cast<float*>(abuf);  // [wave][row]; the last step's barrier has passed
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float v = 0.0f;
#pragma unroll
          for (int n = 0; n < NT; ++n) v = fmaxf(v, fabsf(acc[m][n][r]));
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
          if (fr == 0) rowmax[wave * MR + 16 * m + 4 * g + r] = v;
        }
      __syncthreads();
      const int nyb = (a.N + kYBlock - 1) / kYBlock;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int p = row_of(m, r);
          float v = rowmax[16 * m + 4 * g + r];
#pragma unroll
          for (int w = 1; w < kQrWaves; ++w) v = fmaxf(v, rowmax[w * MR + 16 * m + 4 * g + r]);
          const int e = yexp_of(v);
          if (p < blk.end) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (tile0 + n < a.tiles)
                ((_Float16*)a.out)[(size_t)p * a.N + (tile0 + n) * 16 + fr] = (_Float16)ldexpf(acc[m][n][r], -e);
            if (wave == 0 && fr == 0) a.ye[(size_t)p * nyb + col_wg] = (int8_t)e;
          }
        }
    }
  }
  __device__ __forceinline__ void run(int col_wg) {
    sums();
    if constexpr (W13)
      store_h();
    else
      store_y(col_wg);
  }
};

template <typename XT, int FMT, int GPB, bool W13>
__global__ __launch_bounds__(kQrWaves * 64) void q4_rows(Q4Rows a) {
  constexpr int kMaxMT = sizeof(XT) == 2 ? 4 : 2;
  __shared__ __attribute__((aligned(16))) char abuf[2 * kQrLds];
  __shared__ __attribute__((aligned(16))) float xsum[2 * GPB * 16 * kMaxMT];
  const int cols = (a.tiles + kQrColTiles - 1) / kQrColTiles;  // workgroups across the output
  const int col_wg = blockIdx.x % cols;
  const RowBlock blk = find_block<16 * kMaxMT>(a.offsets, a.E, blockIdx.x / cols);
  if (blk.e < 0) return;
  const int mt = (min(blk.end - blk.row0, 16 * kMaxMT) + 15) / 16;  // the same for the whole workgroup
  if (mt == 1) {
    RowsBody<XT, FMT, GPB, 1, W13>(a, blk, col_wg, abuf, xsum).run(col_wg);
  } else if (mt == 2) {
    RowsBody<XT, FMT, GPB, 2, W13>(a, blk, col_wg, abuf, xsum).run(col_wg);
  } else if constexpr (kMaxMT > 2) {
    if (mt == 3)
      RowsBody<XT, FMT, GPB, 3, W13>(a, blk, col_wg, abuf, xsum).run(col_wg);
    else
      RowsBody<XT, FMT, GPB, 4, W13>(a, blk, col_wg, abuf, xsum).run(col_wg);
  }
}

// Launch over every row block (an upper bound of their number is known on the
// host; workgroups past the last exit at once).
template <typename XT, bool W13>
inline hipError_t launch_rows_of(const Shape& s, const Q4& q, const Q4Rows& a, hipStream_t st) {
  constexpr int kRows = sizeof(XT) == 2 ? 64 : 32;
  const long long blocks = s.R() / kRows + (s.R() < s.E ? s.R() : s.E);
  const dim3 grid((unsigned)(blocks * ((a.tiles + kQrColTiles - 1) / kQrColTiles))), block(kQrWaves * 64);
#define Q4_GO(FMT, GPB) hipLaunchKernelGGL((q4_rows<XT, FMT, GPB, W13>), grid, block, 0, st, a)
  if (q.format == kQ4Int) {
    if (q.group == 128) Q4_GO(kQ4Int, 1);
    else if (q.group == 64) Q4_GO(kQ4Int, 2);
    else Q4_GO(kQ4Int, 4);
  } else {
    if (q.group == 128) Q4_GO(kQ4E2m1, 1);
    else if (q.group == 64) Q4_GO(kQ4E2m1, 2);
    else Q4_GO(kQ4E2m1, 4);
  }
#undef Q4_GO
  return hipGetLastError();
}

template <bool W13>
inline hipError_t launch_rows(const Shape& s, const Q4& q, const Q4Rows& a, hipStream_t st) {
  return s.bf16 ? launch_rows_of<uint16_t, W13>(s, q, a, st) : launch_rows_of<float, W13>(s, q, a, st);
}

}  // namespace moe
