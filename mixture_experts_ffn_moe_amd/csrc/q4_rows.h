// Grouped products over 4-bit weights, few rows per expert: one template for
// the gate|up product with SwiGLU and for the down product.
//
// The codes are the bulk of the bytes and each is used once per block of
// rows, so they go from HBM straight to registers in operand order (a wave
// loads whole 1 KB tiles, 16 bytes a lane), one step ahead of their use.  The
// rows' operands (x gathered through perm, or h) are shared by the
// workgroup's waves: 16 KB of them a step through LDS, double-buffered, one
// barrier a step.  A row of 256 bytes (128 columns) keeps its 16-byte chunks
// XOR-swizzled by the row, so the 16 rows of a fragment read hit 16 bank
// groups.
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

template <typename XT, int FMT, int GPB, int MT, int NT, bool W13>
__global__ __launch_bounds__(kQrWaves * 64) void q4_rows(Q4Rows a) {
  constexpr bool kBf16 = sizeof(XT) == 2;
  constexpr int MR = 16 * MT;
  constexpr int KC = 4 / MT;                    // code tiles per step
  constexpr int kRowBytes = kQ4TileK * (int)sizeof(XT);
  constexpr int kChunks = kRowBytes / 16;       // 16-byte chunks of a row's tile
  constexpr int kBuf = KC * MR * kRowBytes;
  constexpr int kLoads = kBuf / 16 / (kQrWaves * 64);
  constexpr bool kSums = kBf16 && FMT == kQ4Int;
  constexpr int JG = 4 / GPB;                   // 32-column pieces per group
  __shared__ __attribute__((aligned(16))) char abuf[2][kBuf];
  __shared__ __attribute__((aligned(16))) float xsum[2][kSums ? KC * GPB * MR : 4];
  __shared__ float rowmax[kQrWaves][MR];

  const int cols = (a.tiles + kQrWaves * NT - 1) / (kQrWaves * NT);  // workgroups across the output
  const int col_wg = blockIdx.x % cols;
  const RowBlock blk = find_block<MR>(a.offsets, a.E, blockIdx.x / cols);
  if (blk.e < 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, g = lane >> 4;
  const int nb = a.segments * a.KB;

  // this wave's output tiles; past the last they repeat it and store nothing
  const int tile0 = (col_wg * kQrWaves + wave) * NT;
  const uint8_t* codes[NT];
  const XT* scales[NT];
  const size_t seg_codes = (size_t)a.E * (a.N / 16) * a.KB * kQ4TileBytes, seg_scales = (size_t)a.E * a.N * a.S;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int ct = min(tile0 + n, a.tiles - 1);
    const int per = a.N / 16;                              // row tiles of one matrix
    const int m = W13 ? ct / per : 0, it = W13 ? ct % per : ct;
    const size_t tile = ((size_t)m * a.E + blk.e) * per + it;
    codes[n] = a.codes + tile * a.KB * kQ4TileBytes + lane * 16;
    scales[n] = (const XT*)a.scales + (tile * 16 + fr) * a.S;
  }

  // the chunks this thread stages: fixed rows, one source pointer each
  const XT* src[kLoads];
  bool row_ok[kLoads];
  int lds_off[kLoads], kbl[kLoads], col[kLoads], sum_at[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int q = tid + i * kQrWaves * 64;
    const int c = q % kChunks, r = q / kChunks % MR;
    kbl[i] = q / (kChunks * MR);
    col[i] = c * (16 / (int)sizeof(XT));
    const int p = blk.row0 + r;
    row_ok[i] = p < blk.end;
    const int pc = min(p, blk.end - 1);
    src[i] = (const XT*)a.x + (size_t)(W13 ? a.perm[pc] / a.k : pc) * a.ldx;
    const int sw = kBf16 ? (r & 15) : (r & 15) << 1;
    lds_off[i] = (kbl[i] * MR + r) * kRowBytes + ((c ^ sw) * 16);
    sum_at[i] = (kbl[i] * GPB + c / (kChunks / GPB)) * MR + r;
  }

  const Q4Consts kc;
  uint4 av[kLoads], cw[KC][NT], cn[KC][NT];
  float sw[KC][NT][GPB], sn[KC][NT][GPB];
  auto load_rows = [&](int b0) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int b = b0 + kbl[i];
      const int seg = W13 ? 0 : b / a.KB;
      const int col0 = (b - seg * a.KB) * kQ4TileK + col[i];  // column within the matrix
      const bool ok = row_ok[i] && b < nb && col0 < a.K;
      // a chunk that is not ok loads the row's first columns and is dropped
      const uint4 v = *reinterpret_cast<const uint4*>(src[i] + (ok ? (size_t)seg * a.K + col0 : 0));
      av[i] = ok ? v : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_codes = [&](int b0, uint4 (&cv)[KC][NT], float (&sv)[KC][NT][GPB]) {
#pragma unroll
    for (int u = 0; u < KC; ++u) {
      const int b = min(b0 + u, nb - 1);  // past the end: loaded again, not used
      const int seg = W13 ? 0 : b / a.KB;
      const int kb = b - seg * a.KB;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        cv[u][n] = *reinterpret_cast<const uint4*>(codes[n] + seg * seg_codes + (size_t)kb * kQ4TileBytes);
        q4_load_scales<GPB>(scales[n] + seg * seg_scales + kb * GPB, sv[u][n]);
      }
    }
  };
  auto store_rows = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      *reinterpret_cast<uint4*>(abuf[buf] + lds_off[i]) = av[i];
      if constexpr (kSums) {
        const uint32_t w[4] = {av[i].x, av[i].y, av[i].z, av[i].w};
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) s += __uint_as_float(w[j] << 16) + __uint_as_float(w[j] & 0xffff0000u);
#pragma unroll
        for (int d = 1; d < kChunks / GPB; d <<= 1) s += __shfl_xor(s, d);
        if ((tid & (kChunks / GPB - 1)) == 0) xsum[buf][sum_at[i]] = -136.0f * s;
      }
    }
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};

  load_rows(0);
  load_codes(0, cw, sw);
  store_rows(0);
  __syncthreads();
  for (int b0 = 0, buf = 0; b0 < nb; b0 += KC, buf ^= 1) {
    const bool more = b0 + KC < nb;
    if (more) {
      load_rows(b0 + KC);
      load_codes(b0 + KC, cn, sn);
    }
#pragma unroll
    for (int u = 0; u < KC; ++u) {
      if (b0 + u < nb) {
#pragma unroll
        for (int gr = 0; gr < GPB; ++gr) {
          f32x4 part[MT][NT];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            f32x4 start = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (kSums) start = *reinterpret_cast<const f32x4*>(&xsum[buf][(u * GPB + gr) * MR + 16 * m + 4 * g]);
#pragma unroll
            for (int n = 0; n < NT; ++n) part[m][n] = start;
          }
#pragma unroll
          for (int jj = 0; jj < JG; ++jj) {
            const int j = gr * JG + jj;
            bf16x8 bv[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t w = j == 0 ? cw[u][n].x : j == 1 ? cw[u][n].y : j == 2 ? cw[u][n].z : cw[u][n].w;
              bv[n] = q4_operand<FMT>(w, kc);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const char* row = abuf[buf] + (u * MR + 16 * m + fr) * kRowBytes;
              if constexpr (kBf16) {
                const bf16x8 av8 = *reinterpret_cast<const bf16x8*>(row + (((4 * j + g) ^ fr) * 16));
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  part[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av8, bv[n], part[m][n], 0, 0, 0);
              } else {
                // fp32 operands: element i of the four lane groups is one k-step of 4
                const int c = 2 * (4 * j + g);
                const f32x4 lo = *reinterpret_cast<const f32x4*>(row + ((c ^ (fr << 1)) * 16));
                const f32x4 hi = *reinterpret_cast<const f32x4*>(row + (((c + 1) ^ (fr << 1)) * 16));
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
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[m][n][r] = fmaf(sw[u][n][gr], part[m][n][r], acc[m][n][r]);
        }
      }
    }
    if (more) {
      store_rows(buf ^ 1);
#pragma unroll
      for (int u = 0; u < KC; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          cw[u][n] = cn[u][n];
#pragma unroll
          for (int q = 0; q < GPB; ++q) sw[u][n][q] = sn[u][n][q];
        }
    }
    __syncthreads();
  }

  // D layout: register r of a lane holds row 4 (lane/16) + r, column lane%16
  if constexpr (W13) {
    // tile columns 0-7 gate, 8-15 the up columns of the same 8
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int ct = tile0 + n;
      const int per = a.N / 16;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float up = __shfl_xor(acc[m][n][r], 8);
          const int p = blk.row0 + 16 * m + 4 * g + r;
          if (ct < a.tiles && fr < 8 && p < blk.end)
            ((XT*)a.out)[(size_t)p * (a.tiles * 8) + (ct / per) * a.Im + (ct % per) * 8 + fr] =
                Elem<XT>::from_f(silu_f32(acc[m][n][r]) * up);
        }
    }
  } else if constexpr (!kBf16) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int p = blk.row0 + 16 * m + 4 * g + r;
          if (tile0 + n < a.tiles && p < blk.end)
            ((float*)a.out)[(size_t)p * a.N + (tile0 + n) * 16 + fr] = acc[m][n][r];
        }
  } else {
    // block-scaled half y: the workgroup's columns are one block of 256
    // (repeated tiles past H repeat a stored column: the maximum is unchanged)
    static_assert(W13 || !kBf16 || kQrWaves * NT * 16 == kYBlock, "one y block per workgroup");
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) v = fmaxf(v, fabsf(acc[m][n][r]));
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
        if (fr == 0) rowmax[wave][16 * m + 4 * g + r] = v;
      }
    __syncthreads();
    const int nyb = (a.N + kYBlock - 1) / kYBlock;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * m + 4 * g + r, p = blk.row0 + row;
        float v = rowmax[0][row];
#pragma unroll
        for (int w = 1; w < kQrWaves; ++w) v = fmaxf(v, rowmax[w][row]);
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

// Rows per block by the average rows of an expert.
inline int q4_row_tiles(const Shape& s) {
  if (!s.bf16) return 2;
  const long long avg = s.R() / s.E;
  return avg <= 12 ? 1 : avg <= 28 ? 2 : 4;
}

// Launch over every row block (an upper bound of their number is known on the
// host; workgroups past the last exit at once).
template <typename XT, int MT, int NT, bool W13>
inline hipError_t launch_rows_mt(const Shape& s, const Q4& q, const Q4Rows& a, hipStream_t st) {
  const long long blocks = (s.R() / (16 * MT)) + (s.R() < s.E ? s.R() : s.E);
  const dim3 grid((unsigned)(blocks * ((a.tiles + kQrWaves * NT - 1) / (kQrWaves * NT)))), block(kQrWaves * 64);
#define Q4_GO(FMT, GPB) hipLaunchKernelGGL((q4_rows<XT, FMT, GPB, MT, NT, W13>), grid, block, 0, st, a)
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
  if (!s.bf16) return launch_rows_mt<float, 2, 2, W13>(s, q, a, st);
  const int mt = q4_row_tiles(s);
  if (mt == 1) return launch_rows_mt<uint16_t, 1, 2, W13>(s, q, a, st);
  if (mt == 2) return launch_rows_mt<uint16_t, 2, 2, W13>(s, q, a, st);
  return launch_rows_mt<uint16_t, 4, 2, W13>(s, q, a, st);
}

}  // namespace moe
