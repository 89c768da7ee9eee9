// Tiled matrix products of the shared expert's training step and of its
// request adapters (gfx950).
//
//   C[m, n] = sum_k A(m, k) B(n, k),  bf16 or fp32 elements, fp32 sums.
//
// Either operand is stored with k contiguous (rows of k: x, weights in the
// forward pass) or with k as the row index ("k-rows": weights where the
// gradient runs back through them, both operands of a weight gradient).
//   * global -> LDS copies are direct (dma16), a ring of SLOTS k-tiles of KB
//     bytes of k a row.  A k-contiguous tile holds KB-byte rows whose 16-byte
//     chunks are XOR-swizzled by row; a k-rows tile holds BK rows of the
//     tile's columns, swizzled in units of 16 columns.
//   * operands of k-rows tiles are transposed on the way out of LDS: bf16 by
//     the transposing 8-byte read (16 lanes give the addresses of four rows
//     of 16 columns, lane i receives column i of the four rows), fp32 by
//     4-byte reads.  No transposed copy of anything is ever written.
//   * the second matrix operand is A, so a lane holds consecutive columns n
//     of one row m; the finished tile passes through LDS in strips of F rows
//     per wave (the wave's own region: no workgroup barrier) and each lane
//     finishes 8 consecutive columns with 16-byte loads and stores.
//   * eight waves of 128 x 64 of a 256 x 256 tile (two a SIMD) rather than four of
//     128 x 128 (one): 210 against 220 us for 8192 x 4096 x 4096 both
//     k-contiguous (1.31 PFLOP/s), 204 against 216 us both k-rows; without copies
//     170 us.  Copies and operand reads share LDS; the matrix pipe is busy 80 %
//     of the CUs' cycles at sums of 4096 and 8192, 54 % at 2048, where what a
//     tile does before and behind its sum (9 us a round) weighs more.
//   * small tiles are bound by the copies: 32 x 64 move 29 (one workgroup a CU)
//     to 40 bytes a clock and CU, the direct copies' limit.
// Every row, column and k index that would lie outside an operand is clamped
// to its last one; what was read for them is masked (k) or never stored.
#pragma once

#include "moe_common.h"
#include "tile_choice.h"

namespace moe {
namespace tile {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Matrix instruction for F x F blocks: SUB k-values of one call, 16 bytes of
// each operand a lane (row lane % F, 16-byte chunk lane / F of the SUB values).
template <class E, int F>
struct Mma;
template <>
struct Mma<uint16_t, 32> {
  typedef bf16x8 frag;
  typedef f32x16 acc;
  static constexpr int SUB = 16;
  static __device__ __forceinline__ acc mul(frag a, frag b, acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mma<uint16_t, 16> {
  typedef bf16x8 frag;
  typedef f32x4 acc;
  static constexpr int SUB = 32;
  static __device__ __forceinline__ acc mul(frag a, frag b, acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mma<float, 16> {
  typedef f32x4 frag;
  typedef f32x4 acc;
  static constexpr int SUB = 16;
  // call s contracts the k-values 4 * (lane / 16) + s of both operands
  static __device__ __forceinline__ acc mul(frag a, frag b, acc c) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    return c;
  }
};

// Operand of a product: rows (of k) or, k-rows, columns of a [K, count] matrix.
struct Operand {
  const void* p;
  int ld;     // elements between rows
  int count;  // rows m (or n), k-rows: columns
};

template <class E_, int BM_, int BN_, int WM_, int WN_, int F_, int KB_, int SLOTS_, bool TA_, bool TB_>
struct Cfg {
  typedef E_ E;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, F = F_, SLOTS = SLOTS_;
  static constexpr int KB = KB_;  // bytes of k of a k-tile's row
  static constexpr bool TA = TA_, TB = TB_;  // operand stored as k-rows
  typedef Mma<E, F> M;
  static constexpr int ES = sizeof(E), BK = KB / ES, EPC = 16 / ES;  // elements of a 16-byte chunk
  static constexpr int NW = WM * WN, NTHR = NW * 64;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / F, FN = TN / F;
  static constexpr int NSUB = BK / M::SUB, CPS = 64 / F;  // substeps of a k-tile, chunks of a substep
  static constexpr int AQ = BM * KB / 1024 / NW, BQ = BN * KB / 1024 / NW;  // 1 KB copies a wave makes of a k-tile
  static constexpr int A_BYTES = BM * KB, B_BYTES = BN * KB, SLOT_BYTES = A_BYTES + B_BYTES;
  static constexpr int STRIP_LD = TN + 4;  // floats
  static constexpr int STRIP_BYTES = F * STRIP_LD * 4;
  static constexpr int LDS_BYTES = SLOTS * SLOT_BYTES > NW * STRIP_BYTES ? SLOTS * SLOT_BYTES : NW * STRIP_BYTES;
  static_assert(BM * KB % (1024 * NW) == 0 && BN * KB % (1024 * NW) == 0 && TM % F == 0 && TN % F == 0, "tile split");
  static_assert(SLOTS >= 2 && (SLOTS - 2) * (AQ + BQ) < 64, "vmcnt");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

// Swizzle of a k-contiguous tile: 16 rows read together hit 16 distinct
// 16-byte slots of the 256 bytes that LDS serves at once.
template <int KB>
__device__ __forceinline__ int swz_row(int row) {
  static_assert(KB == 128 || KB == 64, "row bytes");
  return KB == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
}

// Swizzle of a k-rows tile of C columns: XOR of the 16-column unit of row k,
// below the number of units of a row.  32 lanes of a bf16 read take four rows
// (F = 32: of two adjacent units) or eight (F = 16: k and k + 8, of one unit);
// the XOR sends them to the eight 32-byte slots of 256 bytes.  fp32 reads take
// four rows, four apart (two of them meet where a row has two units only).
template <class E, int F, int C>
__device__ __forceinline__ int swz_k(int k) {
  static_assert(C >= 128 || C == 64 || (C == 32 && F == 16), "units of a row");
  if (sizeof(E) == 4) return (k >> 2) & (C >= 64 ? 3 : 1);
  if (F == 32) return C >= 128 ? (k & 3) << 1 : k & 2;
  return C >= 128 ? (k & 3) | ((k >> 1) & 4) : C == 64 ? ((k >> 1) & 1) | ((k >> 2) & 2) : (k >> 3) & 1;
}

// Source byte offsets of a wave's direct copies of one operand tile, relative
// to the tile's base (the first row's, k-rows: first column's, at the current
// k-tile).  C rows or columns from `first`, at most `count` of them exist.
// row_of: stored row, relative to the base, of the tile's row (not for k-rows).
// k_left: k-values from the k-tile's start to the end of K.
template <class C, bool KROWS, int N, int Q, class Row>
__device__ __forceinline__ void copy_offsets(uint32_t (&off)[Q], int first, int count, int ld, int k_left,
                                             int wave, int lane, Row row_of) {
  typedef typename C::E E;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = wave + C::NW * i;
    if (!KROWS) {
      constexpr int CPR = C::KB / 16;  // chunks of a row
      const int row = q * (64 / CPR) + lane / CPR;
      int c = (lane % CPR) ^ swz_row<C::KB>(row);
      if (c * C::EPC >= k_left) c = 0;
      off[i] = ((uint32_t)row_of(row) * (uint32_t)ld + (uint32_t)(c * C::EPC)) * C::ES;
    } else {
      constexpr int CPR = N * C::ES / 16;  // chunks of a k-row
      constexpr int UC = C::ES;            // chunks of a 16-column unit
      const int k = q * (64 / CPR) + lane / CPR;
      const int c = lane % CPR;
      int n = (((c / UC) ^ swz_k<E, C::F, N>(k)) * UC + c % UC) * C::EPC;
      n = min(n, count - first - C::EPC);
      off[i] = ((uint32_t)min(k, k_left - 1) * (uint32_t)ld + (uint32_t)n) * C::ES;
    }
  }
}

// Operand fragment of substep ks from an LDS tile: rows r0 .. r0 + F.
template <class C, bool KROWS, int N>
__device__ __forceinline__ typename C::M::frag read_frag(const char* t, int r0, int ks, int lane) {
  typedef typename C::E E;
  if constexpr (!KROWS) {
    const int row = r0 + lane % C::F;
    const int c = (ks * C::CPS + lane / C::F) ^ swz_row<C::KB>(row);
    return *reinterpret_cast<const typename C::M::frag*>(t + row * C::KB + c * 16);
  } else if constexpr (C::ES == 2) {
    const int g = lane >> 4, i = lane & 15;
    const int unit = r0 / 16 + (C::F == 32 ? (g & 1) : 0);
    const int k0 = ks * C::M::SUB + 8 * (C::F == 32 ? g >> 1 : g) + (i >> 2);
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    union {
      s16x4 h[2];
      bf16x8 v;
    } u;
    const char* a = t + k0 * (N * 2) + ((unit ^ swz_k<E, C::F, N>(k0)) * 32) + (i & 3) * 8;
    // k0 + 4 has the same swizzle
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a));
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * (N * 2)));
    return u.v;
  } else {
    const int k0 = ks * C::M::SUB + 4 * (lane >> 4);
    f32x4 v;
    const char* a = t + k0 * (N * 4) + ((r0 / 16) ^ swz_k<E, C::F, N>(k0)) * 64 + (lane & 15) * 4;
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = *reinterpret_cast<const float*>(a + s * (N * 4));
    return v;
  }
}

// Zeroes the k-values at and past `left` (k-values from the substep's start).
template <class C>
__device__ __forceinline__ typename C::M::frag mask_k(typename C::M::frag f, int left, int lane) {
  constexpr int N = 16 / C::ES;
  const int mine = left - N * (lane / C::F);
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (e >= mine) f[e] = 0.0f;
  return f;
}

__device__ __forceinline__ void slot_barrier() {
  __builtin_amdgcn_s_waitcnt(0xF | (7 << 4) | (0 << 8) | (3 << 14));  // lgkmcnt(0)
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Wait states between a matrix instruction and the first vector instruction
// that reads its result, where a branch lies between them: the compiler counts
// them within a block only.
__device__ __forceinline__ void settle() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15");
  __builtin_amdgcn_sched_barrier(0);
}

// Tile t of mt x nt: tiles run down groups of four row tiles, so that the 32
// tiles a die works on at a time (4 x 8) share their rows and columns in its L2.
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int& m, int& n) {
  constexpr int G = 4;
  const int group = t / (G * nt), in = t - group * (G * nt);
  const int rows = min(G, mt - group * G);
  m = group * G + in % rows;
  n = in / rows;
}

// No low-rank addition.
struct NoExtra {
  static constexpr bool ON = false, MAPPED = false;
  __device__ __forceinline__ int a_row(int r) const { return r; }
  __device__ __forceinline__ int out_row(int r) const { return r; }
  template <class C, class R0, class Row>
  __device__ __forceinline__ int begin(int, int, R0, Row, int, int) const { return 0; }
};

// One tile, from row m0 and column n0 on.  PAIR: B has two halves of `half`
// rows (gate, up) and a tile takes BN / 2 columns of each; the epilogue then
// gets both values of a column.
template <class C, class Epi, class Extra>
__device__ __forceinline__ void product(const Operand A, const Operand B, int K, int half, int m0, int n0,
                                        const Epi& epi, const Extra& extra, char* smem) {
  constexpr bool PAIR = Epi::PAIR;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int N = PAIR ? half : B.count;
  const int KT = (K + C::BK - 1) / C::BK;

  // bases of the tile (k-tile 0) and the row maps below them
  constexpr bool rowmap = Extra::MAPPED;  // rows of A are gathered
  const char* a0 = (const char*)A.p + (C::TA ? (size_t)m0 : rowmap ? 0 : (size_t)m0 * A.ld) * C::ES;
  const char* b0 = (const char*)B.p + (C::TB ? (size_t)n0 : PAIR ? 0 : (size_t)n0 * B.ld) * C::ES;
  auto arow = [&](int r) {
    const int g = min(m0 + r, A.count - 1);
    return rowmap ? extra.a_row(g) : g - m0;
  };
  auto brow = [&](int r) {
    if (!PAIR) return min(n0 + r, B.count - 1) - n0;
    const int up = r >= C::BN / 2;
    return up * half + min(n0 + r - up * (C::BN / 2), half - 1);
  };
  const size_t a_step = C::TA ? (size_t)C::BK * A.ld * C::ES : (size_t)C::KB;
  const size_t b_step = C::TB ? (size_t)C::BK * B.ld * C::ES : (size_t)C::KB;
  uint32_t aoff[C::AQ], boff[C::BQ];
  copy_offsets<C, C::TA, C::BM>(aoff, m0, A.count, A.ld, K, wave, lane, arow);
  copy_offsets<C, C::TB, C::BN>(boff, n0, B.count, B.ld, K, wave, lane, brow);

  const uint32_t lds = (uint32_t)(uintptr_t)smem;
  // Copies: k-tile `next` goes out piece by piece.  Past the last k-tile the
  // last one is copied again (into slots that are not read any more), so that
  // every wait counts the same number of copies.
  int next = 0;
  uint32_t slot = 0;
  const char *pa = nullptr, *pb = nullptr;
  auto copy_begin = [&]() {
    const int kt = min(next, KT - 1);
    if (kt > 0 && next == KT - 1 && K % C::BK != 0) {  // the last k-tile is short
      copy_offsets<C, C::TA, C::BM>(aoff, m0, A.count, A.ld, K - kt * C::BK, wave, lane, arow);
      copy_offsets<C, C::TB, C::BN>(boff, n0, B.count, B.ld, K - kt * C::BK, wave, lane, brow);
    }
    slot = lds + (uint32_t)((next % C::SLOTS) * C::SLOT_BYTES);
    pa = uniform_ptr(a0 + kt * a_step);
    pb = uniform_ptr(b0 + kt * b_step);
    ++next;
  };
  auto copy_piece = [&](int i) {
    if (i < C::AQ)
      dma16(slot + (uint32_t)(wave + C::NW * i) * 1024u, pa, aoff[i]);
    else
      dma16(slot + C::A_BYTES + (uint32_t)(wave + C::NW * (i - C::AQ)) * 1024u, pb, boff[i - C::AQ]);
  };
  constexpr int NI = C::AQ + C::BQ;

  typename C::M::acc acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int e = 0; e < C::F * C::F / 64; ++e) acc[i][j][e] = 0.0f;

  auto b_r0 = [&](int j) {
    if (!PAIR) return wn * C::TN + C::F * j;
    return j < C::FN / 2 ? wn * (C::TN / 2) + C::F * j : C::BN / 2 + wn * (C::TN / 2) + C::F * (j - C::FN / 2);
  };
  static_assert(!PAIR || C::FN % 2 == 0, "gate and up fragments of a wave");

  if (KT > 0) {
    for (int s = 0; s < C::SLOTS - 1; ++s) {
      copy_begin();
#pragma unroll
      for (int i = 0; i < NI; ++i) copy_piece(i);
    }
  }
  auto all_row = [&](int r) {  // row of B, from its start, of tile row r
    const int up = PAIR && r >= C::BN / 2;
    return up * half + min(n0 + r - up * (C::BN / 2), N - 1);
  };
  [[maybe_unused]] const auto ahead = extra.template begin<C>(m0, wm * C::TM, b_r0, all_row, wave, lane);
  // The next k-tile has landed for every wave, and the slot of the one before it is free.
  auto landed = [&]() {
    wait_vmcnt<(C::SLOTS - 2) * NI>();
    slot_barrier();
  };
  struct Frags {
    typename C::M::frag a[C::FM], b[C::FN];
  };
  // Fragment q of a substep, in the order in which products need them.
  constexpr int NF = C::FM + C::FN;
  auto read = [&](Frags& f, int q, const char* ta, int ks) {
    if (q >= 1 && q <= C::FN)
      f.b[q - 1] = read_frag<C, C::TB, C::BN>(ta + C::A_BYTES, b_r0(q - 1), ks, lane);
    else {
      const int i = q ? q - C::FN : 0;
      f.a[i] = read_frag<C, C::TA, C::BM>(ta, wm * C::TM + C::F * i, ks, lane);
    }
  };
  auto tile_at = [&](int kt) { return smem + (kt % C::SLOTS) * C::SLOT_BYTES; };
  // Products n0 .. n1 of a substep's FM x FN.  Behind every product goes a read
  // of the next substep's operands (RPP of them, as long as there are any), then copies p0 .. p1,
  // spread over the products that are left: a wave issues in order, and a
  // run of reads or copies would fill their queue and hold up the products
  // behind it.
  constexpr int NP = C::FM * C::FN, RPP = (2 * NF + NP - 1) / NP;
  auto multiply = [&](const Frags& f, int n0, int n1, Frags* into, const char* ta, int ks, int p0, int p1) {
    const int rn = into ? (NF + RPP - 1) / RPP : 0;          // products that carry reads
    const int cn = n1 - n0 - rn > 0 ? n1 - n0 - rn : 1;      // products that may carry copies
#pragma unroll
    for (int n = n0; n < n1; ++n) {
      const int i = n / C::FN, j = n % C::FN;
      acc[i][j] = C::M::mul(f.b[j], f.a[i], acc[i][j]);
      if (into) {
#pragma unroll
        for (int q = (n - n0) * RPP; q < (n - n0 + 1) * RPP; ++q)
          if (q < NF) read(*into, q, ta, ks);
        if (n == n1 - 1)
#pragma unroll
          for (int q = (n - n0 + 1) * RPP; q < NF; ++q) read(*into, q, ta, ks);
      }
#pragma unroll
      for (int p = p0; p < p1; ++p)
        if (n1 - cn + (p - p0) * cn / (p1 - p0) == n) copy_piece(p);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // The operands of a substep are read while the one before it multiplies; the
  // last substep of a k-tile has a quarter of its products issued before the
  // wait for the next k-tile.  A k-tile's copies lie between the products of
  // the k-tile SLOTS - 1 before it.
  const int KF = K / C::BK;
  static_assert(C::NSUB % 2 == 0, "substeps in pairs");
  Frags f[2];
  if (KF > 0) {
    landed();
#pragma unroll
    for (int q = 0; q < NF; ++q) read(f[0], q, tile_at(0), 0);
    for (int kt = 0; kt < KF; ++kt) {
      copy_begin();
      const char* ta = tile_at(kt);
#pragma unroll
      for (int ks = 0; ks + 1 < C::NSUB; ++ks)
        multiply(f[ks & 1], 0, NP, &f[(ks + 1) & 1], ta, ks + 1, NI * ks / (C::NSUB - 1), NI * (ks + 1) / (C::NSUB - 1));
      multiply(f[1], 0, NP / 4, nullptr, nullptr, 0, 0, 0);
      landed();
      // past the last whole k-tile the reads fetch what is in the ring and nothing uses it
      multiply(f[1], NP / 4, NP, &f[0], tile_at(kt + 1), 0, 0, 0);
    }
  }
  if (KF < KT) {
    if (KF == 0) landed();
    const int left = K - KF * C::BK;
    for (int ks = 0; ks * C::M::SUB < left; ++ks) {
      Frags& t = f[0];
#pragma unroll
      for (int q = 0; q < NF; ++q) read(t, q, tile_at(KF), ks);
#pragma unroll
      for (int i = 0; i < C::FM; ++i) t.a[i] = mask_k<C>(t.a[i], left - ks * C::M::SUB, lane);
#pragma unroll
      for (int j = 0; j < C::FN; ++j) t.b[j] = mask_k<C>(t.b[j], left - ks * C::M::SUB, lane);
      multiply(t, 0, NP, nullptr, nullptr, 0, 0, 0);
    }
  }
  settle();
  wait_vmcnt<0>();  // copies that nothing waited for
  __syncthreads();  // every wave is past its last LDS read: the ring is free
  if constexpr (Extra::ON) {
    extra.template add<C>(acc, ahead, smem, m0, wm * C::TM, b_r0, all_row, wave, lane);
    settle();
    __syncthreads();
  }
  float* strip = reinterpret_cast<float*>(smem + wave * C::STRIP_BYTES);
  constexpr int WC = PAIR ? C::TN / 2 : C::TN;  // output columns of the wave
  constexpr int LPR = WC / 8, RPI = 64 / LPR;   // lanes of a row, rows of an iteration
  constexpr int ITER = (C::F + RPI - 1) / RPI;   // RPI > F: the last lanes have no row
  static_assert(WC % 8 == 0 && 64 % LPR == 0 && (C::F % RPI == 0 || RPI % C::F == 0), "epilogue split");
  const int c8 = (lane % LPR) * 8, col = n0 + wn * WC + c8;
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int q = 0; q < C::F * C::F / 256; ++q) {
        const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        *reinterpret_cast<f32x4*>(strip + (lane % C::F) * C::STRIP_LD + C::F * j + 8 * q + 4 * (lane / C::F)) = v;
      }
    __builtin_amdgcn_wave_barrier();
    typename Epi::Pre pre[ITER];
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int r = it * RPI + lane / LPR, row = m0 + wm * C::TM + C::F * i + r;
      if (r < C::F && row < A.count && col < N) pre[it] = epi.load(extra.out_row(row), col);
    }
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int r = it * RPI + lane / LPR, row = m0 + wm * C::TM + C::F * i + r;
      const float* s = strip + (RPI > C::F ? r % C::F : r) * C::STRIP_LD + c8;
      f32x4 v[4];
      v[0] = *reinterpret_cast<const f32x4*>(s);
      v[1] = *reinterpret_cast<const f32x4*>(s + 4);
      if (PAIR) {
        v[2] = *reinterpret_cast<const f32x4*>(s + WC);
        v[3] = *reinterpret_cast<const f32x4*>(s + WC + 4);
      }
      if (r < C::F && row < A.count && col < N) epi.store(extra.out_row(row), col, v, pre[it]);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Block b runs on die b % 8; each die takes a contiguous range of tiles.
template <class C, class Epi, class Extra>
__global__ __launch_bounds__(C::NTHR, 1) void product_kernel(Operand A, Operand B, int K, int half, int mt, int nt,
                                                             Epi epi, Extra extra) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS_BYTES];
  const int all = mt * nt, per = (all + kXcds - 1) / kXcds;
  const int slot = blockIdx.x / kXcds, t = (blockIdx.x % kXcds) * per + slot;
  if (slot >= per || t >= all) return;
  int tm, tn;
  tile_of(t, mt, nt, tm, tn);
  product<C, Epi, Extra>(A, B, K, half, tm * C::BM, tn * (Epi::PAIR ? C::BN / 2 : C::BN), epi, extra, smem);
}

template <class C, class Epi, class Extra>
hipError_t launch_product(Operand A, Operand B, int K, int half, const Epi& epi, hipStream_t st, const Extra& extra) {
  const int oc = Epi::PAIR ? C::BN / 2 : C::BN, N = Epi::PAIR ? half : B.count;
  const int mt = (A.count + C::BM - 1) / C::BM, nt = (N + oc - 1) / oc;
  const unsigned grid = (unsigned)(((long long)mt * nt + kXcds - 1) / kXcds * kXcds);
  hipLaunchKernelGGL((product_kernel<C, Epi, Extra>), dim3(grid), dim3(C::NTHR), 0, st, A, B, K, half, mt, nt, epi,
                     extra);
  return hipGetLastError();
}

// The tile sizes a product may take (tile_choice.h).
template <class E, int I, bool TA, bool TB>
struct TileCfg;
template <bool TA, bool TB> struct TileCfg<uint16_t, 0, TA, TB> { typedef Cfg<uint16_t, 32, 64, 2, 2, 16, 128, 4, TA, TB> type; };
template <bool TA, bool TB> struct TileCfg<uint16_t, 1, TA, TB> { typedef Cfg<uint16_t, 64, 64, 2, 2, 16, 128, 4, TA, TB> type; };
template <bool TA, bool TB> struct TileCfg<uint16_t, 2, TA, TB> { typedef Cfg<uint16_t, 64, 128, 2, 4, 16, 128, 4, TA, TB> type; };
template <bool TA, bool TB> struct TileCfg<uint16_t, 3, TA, TB> { typedef Cfg<uint16_t, 128, 128, 2, 2, 32, 128, 4, TA, TB> type; };
template <bool TA, bool TB> struct TileCfg<uint16_t, 4, TA, TB> { typedef Cfg<uint16_t, 128, 256, 2, 4, 32, 128, 3, TA, TB> type; };
template <bool TA, bool TB> struct TileCfg<uint16_t, 5, TA, TB> { typedef Cfg<uint16_t, 256, 256, 2, 4, 32, 64, 4, TA, TB> type; };
template <bool TA, bool TB> struct TileCfg<float, 0, TA, TB> { typedef Cfg<float, 32, 64, 2, 2, 16, 128, 4, TA, TB> type; };
template <bool TA, bool TB> struct TileCfg<float, 1, TA, TB> { typedef Cfg<float, 64, 64, 4, 2, 16, 128, 4, TA, TB> type; };
template <bool TA, bool TB> struct TileCfg<float, 2, TA, TB> { typedef Cfg<float, 128, 128, 2, 4, 16, 128, 4, TA, TB> type; };

// f(index constant) for tile size i.
template <int I>
struct Index {
  static constexpr int value = I;
};
template <class E, int I = 0, class F>
hipError_t with_tile(int i, F f) {
  if constexpr (I + 1 < TileCosts<E>::COUNT)
    if (i != I) return with_tile<E, I + 1>(i, f);
  return f(Index<I>{});
}
// The product with the tile size that is estimated to be the fastest.
template <class E, bool TA, bool TB, class Epi, class Extra = NoExtra>
hipError_t run_product(const Operand& A, const Operand& B, int K, int half, const Epi& epi, hipStream_t st,
                       const Extra& extra = Extra{}) {
  const int i = product_tile<E>(A.count, Epi::PAIR ? 2ll * half : B.count, K);
  return with_tile<E>(i, [&](auto index) {
    return launch_product<typename TileCfg<E, decltype(index)::value, TA, TB>::type>(A, B, K, half, epi, st, extra);
  });
}

// ---------------------------------------------------------------------------
// Eight consecutive elements of a row: one 16-byte vector of bf16, two of fp32.
template <class E>
struct Vec8;
template <>
struct Vec8<uint16_t> {
  uint4 d;
  __device__ __forceinline__ void load(const uint16_t* p) { d = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t w = i < 2 ? d.x : i < 4 ? d.y : i < 6 ? d.z : d.w;
    return (i & 1) ? __uint_as_float(w & 0xffff0000u) : __uint_as_float(w << 16);
  }
};
template <>
struct Vec8<float> {
  f32x4 d[2];
  __device__ __forceinline__ void load(const float* p) {
    d[0] = reinterpret_cast<const f32x4*>(p)[0];
    d[1] = reinterpret_cast<const f32x4*>(p)[1];
  }
  __device__ __forceinline__ float operator[](int i) const { return d[i >> 2][i & 3]; }
};
__device__ __forceinline__ void store8(uint16_t* p, f32x4 a, f32x4 b) {
  const uint2 lo = pack_bf16x4(a), hi = pack_bf16x4(b);
  *reinterpret_cast<uint4*>(p) = make_uint4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ void store8(float* p, f32x4 a, f32x4 b) {
  reinterpret_cast<f32x4*>(p)[0] = a;
  reinterpret_cast<f32x4*>(p)[1] = b;
}

// out[row, col] = v (+ residual)
template <class E>
struct StoreOut {
  static constexpr bool PAIR = false;
  E* out;
  const E* residual;  // may be null
  int ld;
  struct Pre {
    Vec8<E> r;
  };
  __device__ __forceinline__ Pre load(int row, int col) const {
    Pre p;
    if (residual) p.r.load(residual + (size_t)row * ld + col);
    return p;
  }
  __device__ __forceinline__ void store(int row, int col, f32x4* v, const Pre& p) const {
    if (residual) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] += p.r[i];
    }
    store8(out + (size_t)row * ld + col, v[0], v[1]);
  }
};

}  // namespace tile
}  // namespace moe
