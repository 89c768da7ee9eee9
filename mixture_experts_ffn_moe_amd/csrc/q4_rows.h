// Grouped products over 4-bit weights: one template for the gate|up product
// with SwiGLU and for the down product.
//
// A workgroup of 8 waves takes up to 48 rows of one expert (16 MT, MT the
// fewest 16-row tiles that hold them; fp32 32) and 256 weight rows, a wave 32 of
// them (fp32 half as many).
// The codes are the bulk of the bytes and each is used once per row block, so
// they go from HBM straight to registers in operand order (a wave loads whole
// 1 KB tiles, 16 bytes a lane), four steps of 128 columns ahead of their use.
// The rows' operands (x gathered through perm, or h) are shared by the waves
// and go straight to LDS, as far ahead, in four slots, one barrier a step.
// (Loads return in order: were the rows asked for later than the codes,
// waiting for them would wait for every code in flight.)  A row of 256 bytes
// (128 columns) has its 16-byte chunks XOR-swizzled by the row on the way, so
// the 16 rows of a fragment read hit 16 bank groups.
//
// A row's scales are neighbours along K, so one step needs a few bytes of every
// row's own line.  Four steps' scales are therefore loaded at once, each of the
// four lane groups taking one step's, and handed to the other groups by a lane
// permutation.  (Loaded step by step they were fetched anew each time, more
// lines than the L1 holds: 168 against 144 us for the gate|up product at 256
// tokens, two micro-shards.)
//
// Bound: 256 tokens of the layer H = 4096, E = 64, k = 8, two micro-shards of 768,
// INT4, group 64: the gate|up product takes 134 - 140 us for 430 MB (3.1 - 3.2 TB/s),
// the down product 77 - 81 us for 215 MB; without its products the first takes 95 -
// 112 us, with its codes from the L2 128 us.  What bounds it is the length of a step in a
// wave (operands from LDS, conversion, products, scales) at 16 waves a CU, which
// 128 registers a lane allow (at groups of 128 the gate|up product spills six of them
// in INT4 and one in E2M1, at groups of 64 the INT4 down product one, outside the steps).
// Every block of rows reads and converts all codes of its expert again: past some 1500
// tokens of this layer (of one or two shards) the dense bf16 layer is the faster one.  Tried and not kept: row sums behind the products,
// workgroups of one expert on one XCD, halved workgroups in the last round.
//
// INT4 codes enter as 128 + code (q4.h).  The 136 * sum(x) too much of a
// group is the same for every weight row: each wave sums the chunks that it
// copied itself (8 values on the two-element dot product, then over the group's
// lanes), and -136 times the sum starts the group's accumulator: no extra
// matrix instruction.
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

// Weight row tiles of a wave.  fp32 is bound by its matrix instructions, not by
// the codes: one tile spreads them over more workgroups and needs no spills (37
// tokens of H = 448, seven experts of two shards of 160: 15 + 14 against 25 + 23
// us; 1024 tokens, H = 1024, Im = 512, E = 16, k = 4: 108 + 56 against 133 + 69 us).
template <typename XT>
constexpr int kQrTiles = sizeof(XT) == 2 ? 2 : 1;
template <typename XT>
constexpr int kQrColTiles = kQrWaves * kQrTiles<XT>;
constexpr int kQrLds = 65536;       // bytes of the staged rows' slots, at most

// One direct-to-LDS load of 16 bytes a lane from a 64-bit address (rows whose
// offsets pass 32 bits); otherwise as dma16.
__device__ __forceinline__ void dma16_at(uint32_t lds, const void* p) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :: "s"(lds), "v"(p) : "memory", "m0");
#pragma clang diagnostic pop
}

// All but the N newest loads have arrived, LDS copies among them.
template <int N>
__device__ __forceinline__ void q4_arrived() {
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<N>();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <typename XT, int FMT, int GPB, int MT, bool W13>
struct RowsBody {
  static constexpr bool kBf16 = sizeof(XT) == 2;
  static constexpr int NT = kQrTiles<XT>;
  static constexpr int MR = 16 * MT;
  static constexpr int D = 4;                          // steps in flight, and of one set of scales
  static constexpr int kRowBytes = kQ4TileK * (int)sizeof(XT);
  static constexpr int kChunks = kRowBytes / 16;       // 16-byte chunks of a row's tile
  // copies of 64 chunks that each wave makes per step: 32 or 64 rows (rows past
  // the block repeat its last)
  static constexpr int kCopies = (MT <= 2 ? 32 : 64) * kChunks / 64 / kQrWaves;
  static constexpr int kSlot = kCopies * kQrWaves * 1024;
  static constexpr int kSumRows = MT <= 2 ? 32 : 64;
  static constexpr bool kSums = kBf16 && FMT == kQ4Int;
  static constexpr int JG = 4 / GPB;                   // 32-column pieces per group
  static constexpr int kScaleBytes = GPB * (int)sizeof(XT);
  static constexpr int SW = (kScaleBytes + 3) / 4;     // words of a tile's scales
  static_assert(D * kSlot <= kQrLds, "the slots fit");

  const Q4Rows& a;
  const RowBlock& blk;
  char* abuf;
  float* xsum;    // [slot][group][row]
  const int tid, lane, wave, fr, g, tile0;
  int lseg = 0, lkb = 0;    // the step to load next
  const Q4Consts kc;

  // Addresses are a uniform base (scalar registers) plus a 32-bit offset of the lane.
  const uint8_t* codes[NT];
  const XT* scales[NT];
  size_t seg_codes, seg_scales;
  uint32_t code_off;
  size_t src[kCopies];      // byte offset of the row a copy's lane reads
  int col[kCopies];         // and its column within the tile
  uint4 cw[D][NT];
  uint32_t snext[NT][SW];   // scales of the next D steps, step lane / 16 of them in each lane
  f32x4 acc[MT][NT];

  __device__ __forceinline__ RowsBody(const Q4Rows& a_, const RowBlock& b_, int col_wg, char* abuf_, float* xsum_)
      : a(a_), blk(b_), abuf(abuf_), xsum(xsum_), tid(threadIdx.x), lane(threadIdx.x & 63),
        wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), fr(threadIdx.x & 15), g((threadIdx.x & 63) >> 4),
        tile0((col_wg * kQrWaves + wave) * NT) {
    // this wave's output tiles; past the last they repeat it and store nothing
    seg_codes = (size_t)a.E * (a.N / 16) * a.KB * kQ4TileBytes;
    seg_scales = (size_t)a.E * a.N * a.S;
    const int per = a.N / 16;  // row tiles of one matrix
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int ct = min(tile0 + n, a.tiles - 1);
      const int m = W13 ? ct / per : 0, it = W13 ? ct % per : ct;
      const size_t tile = ((size_t)m * a.E + blk.e) * per + it;
      codes[n] = a.codes + tile * a.KB * kQ4TileBytes;
      scales[n] = (const XT*)a.scales + tile * 16 * a.S;
    }
    code_off = lane * 16;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      // chunk q of the slot holds chunk (q % kChunks) ^ swizzle of row q / kChunks
      const int q = (i * kQrWaves + wave) * 64 + lane, r = q / kChunks;
      const int c = (q % kChunks) ^ (kBf16 ? (r & 15) : (r & 15) << 1);
      const int p = min(blk.row0 + r, blk.end - 1);
      src[i] = (size_t)(W13 ? a.perm[p] / a.k : p) * a.ldx * sizeof(XT);
      col[i] = c * (16 / (int)sizeof(XT));
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // Nontemporal for the gate|up product (256 tokens, two micro-shards: 136
  // against 145 us; T = 64: 54 against 57 us, T = 1024: 188 against 190 us): the
  // rows stay in the L2.  Not for the down product, whose rows are fewer (T =
  // 256: 47 against 48 us, T = 1024: 126 against 130 us).
  //
  // A step is 128 columns, tile kb of segment seg: its rows to the slot, its
  // codes to registers, and on to the step after it.  Past the last step that
  // one is loaded again, and not used.
  __device__ __forceinline__ void next(int slot, uint4 (&c)[NT]) {
    const int kb = lkb, seg = W13 ? 0 : lseg, k0 = kb * kQ4TileK;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      // columns past the matrix meet codes and scales of zero: the row's first columns will do
      const int k = seg * a.K + (k0 + col[i] < a.K ? k0 + col[i] : 0);
      const uint32_t lds = (uint32_t)(uintptr_t)abuf + (uint32_t)(slot * kSlot + (i * kQrWaves + wave) * 1024);
      if constexpr (kBf16)  // fewer than 2^31 elements: offsets below 4 GB
        dma16(lds, a.x, (uint32_t)src[i] + (uint32_t)k * 2u);
      else
        dma16_at(lds, (const char*)a.x + src[i] + (size_t)k * 4);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
      c[n] = load_codes<W13>(codes[n] + seg * seg_codes + (size_t)kb * kQ4TileBytes + code_off);
    const bool wrap = lkb + 1 == a.KB, end = wrap && lseg + 1 == a.segments;
    lkb = end ? lkb : wrap ? 0 : lkb + 1;
    lseg += wrap && !end ? 1 : 0;
  }
  // The scales of the D steps from the next one on, lane group g's of step g
  // (steps past the last: any of the matrix's, not used).
  __device__ __forceinline__ void next_scales() {
    int k = lkb + g, seg = lseg;
    if constexpr (!W13) {
#pragma unroll
      for (int i = 0; i + 1 < D; ++i) {  // a segment may be a single step
        const bool wrap = k >= a.KB && seg + 1 < a.segments;
        k -= wrap ? a.KB : 0;
        seg += wrap ? 1 : 0;
      }
    }
    const size_t off = (W13 ? (size_t)0 : seg * seg_scales) + (size_t)(uint32_t)(fr * a.S + min(k, a.KB - 1) * GPB);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const XT* p = scales[n] + off;
      if constexpr (kScaleBytes == 2) {
        snext[n][0] = *reinterpret_cast<const uint16_t*>(p);
      } else if constexpr (kScaleBytes == 4) {
        snext[n][0] = *reinterpret_cast<const uint32_t*>(p);
      } else if constexpr (kScaleBytes == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        snext[n][0] = v.x;
        snext[n][1] = v.y;
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        snext[n][0] = v.x;
        snext[n][1] = v.y;
        snext[n][2] = v.z;
        snext[n][3] = v.w;
      }
    }
  }
  // Sums of the chunks this wave copied to the slot (they have arrived).
  __device__ __forceinline__ void sum_rows(int slot) const {
    if constexpr (kSums) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int q = (i * kQrWaves + wave) * 64 + lane, r = q / kChunks;
        // the xor swizzle permutes a row's groups and the chunks within one
        const float s = q4_group_start<GPB>(*reinterpret_cast<const uint4*>(abuf + slot * kSlot + q * 16));
        const int c = (lane & 15) ^ (r & 15);
        if ((lane & (16 / GPB - 1)) == 0) xsum[(slot * GPB + c / (16 / GPB)) * kSumRows + r] = s;
      }
    }
  }
  __device__ __forceinline__ float scale(const uint32_t (&s)[SW], int q) const {
    if constexpr (!kBf16) return __uint_as_float(s[q]);
    return __uint_as_float((q & 1) ? s[q / 2] & 0xffff0000u : s[q / 2] << 16);
  }
  __device__ __forceinline__ void products(const uint4 (&c)[NT], const uint32_t (&s)[NT][SW], int slot) {
    const char* rows = abuf + slot * kSlot + fr * kRowBytes;
#pragma unroll
    for (int gr = 0; gr < GPB; ++gr) {
      bf16x8 bv[JG][NT];
      float f[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f[n] = scale(s[n], gr);
#pragma unroll
        for (int jj = 0; jj < JG; ++jj) {
          const int j = gr * JG + jj;
          bv[jj][n] = q4_operand<FMT>(j == 0 ? c[n].x : j == 1 ? c[n].y : j == 2 ? c[n].z : c[n].w, kc);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const char* row = rows + 16 * m * kRowBytes;
        f32x4 part[NT];
        f32x4 start = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (kSums)
          start = *reinterpret_cast<const f32x4*>(&xsum[(slot * GPB + gr) * kSumRows + 16 * m + 4 * g]);
#pragma unroll
        for (int n = 0; n < NT; ++n) part[n] = start;
#pragma unroll
        for (int jj = 0; jj < JG; ++jj) {
          const int j = gr * JG + jj;
          if constexpr (kBf16) {
            const bf16x8 av8 = *reinterpret_cast<const bf16x8*>(row + (((4 * j + g) ^ fr) * 16));
#pragma unroll
            for (int n = 0; n < NT; ++n)
              part[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av8, bv[jj][n], part[n], 0, 0, 0);
          } else {
            // fp32 operands: element i of the four lane groups is one k-step of 4
            const int ch = 2 * (4 * j + g);
            const f32x4 lo = *reinterpret_cast<const f32x4*>(row + ((ch ^ (fr << 1)) * 16));
            const f32x4 hi = *reinterpret_cast<const f32x4*>(row + (((ch + 1) ^ (fr << 1)) * 16));
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                part[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(i < 4 ? lo[i] : hi[i - 4], q4_value<FMT>(bv[jj][n], i),
                                                               part[n], 0, 0, 0);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][n][r] = fmaf(f[n], part[n][r], acc[m][n][r]);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) pin(acc[m][n]);
  }

  // Step d of a set of D, in slot d: once the next step's rows are here, their
  // sums beside this step's products; when every wave is done with the slot,
  // the copies and loads of the step D later into it.  Behind the copies of the
  // next step lie that step's codes and all of the D - 2 steps after it (and,
  // not counted on, a set of scales).
  template <int d, bool kLoad>
  __device__ __forceinline__ void step(const uint32_t (&sset)[NT][SW], bool any) {
    if constexpr (kLoad)
      q4_arrived<NT + (D - 2) * (kCopies + NT)>();
    else
      q4_arrived<0>();
    sum_rows((d + 1) % D);  // past the last step: of an old slot, not used
    if (any) {
      uint32_t s[NT][SW];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int w = 0; w < SW; ++w)
          s[n][w] = (uint32_t)__builtin_amdgcn_ds_bpermute((16 * d + fr) * 4, (int)sset[n][w]);
      products(cw[d], s, d);
    }
    lds_barrier();
    if constexpr (kLoad) next(d, cw[d]);
    __builtin_amdgcn_sched_barrier(0);
  }
  // D steps, `left` of all the steps from the first of them on.
  template <bool kLoad>
  __device__ __forceinline__ void set(int left) {
    uint32_t scur[NT][SW];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int w = 0; w < SW; ++w) scur[n][w] = snext[n][w];
    if constexpr (kLoad) next_scales();
    step<0, kLoad>(scur, true);
    step<1, kLoad>(scur, kLoad || left > 1);
    step<2, kLoad>(scur, kLoad || left > 2);
    step<3, kLoad>(scur, kLoad || left > 3);
  }
  __device__ __forceinline__ void sums() {
    static_assert(D == 4, "set() and the scales' lane groups");
    next_scales();
    next(0, cw[0]);
    next(1, cw[1]);
    next(2, cw[2]);
    next(3, cw[3]);
    q4_arrived<NT + (D - 1) * (kCopies + NT)>();
    sum_rows(0);
    lds_barrier();
    int left = a.segments * a.KB;  // a set may pass from one segment to the next
    for (; left > D; left -= D) set<true>(left);
    set<false>(left);
    __syncthreads();  // the slots are used again; no copy is in flight
  }

  // D layout of the matrix instruction: register r of a lane holds row 4 (lane/16) + r, column lane%16
  __device__ __forceinline__ int row_of(int m, int r) const { return blk.row0 + 16 * m + 4 * g + r; }

  __device__ __forceinline__ void store_h() const {
    // tile columns 0-7 gate, 8-15 the up columns of the same 8; h in the layer's type,
    // as the dense product writes it (the down product's operands are bf16 in bf16 layers)
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
      // block-scaled half y, the dense layer's (11 bits in the bytes of bf16, moe_common.h):
      // the workgroup's columns are one block of 256
      // (repeated tiles past H repeat a stored column: the maximum is unchanged)
      static_assert(kQrColTiles<XT> * 16 == kYBlock, "one y block per workgroup");
      float* rowmax = reinterpret_cast<float*>(abuf);  // [wave][row]
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
__global__ __launch_bounds__(kQrWaves * 64, 4) void q4_rows(Q4Rows a) {  // two workgroups per CU
  constexpr int kMaxMT = sizeof(XT) == 2 ? 3 : 2;
  __shared__ __attribute__((aligned(1024))) char abuf[kQrLds];
  __shared__ __attribute__((aligned(16))) float xsum[4 * GPB * 64];
  const int cols = (a.tiles + kQrColTiles<XT> - 1) / kQrColTiles<XT>;  // workgroups across the output
  const int col_wg = blockIdx.x % cols;
  const RowBlock blk = find_block<16 * kMaxMT>(a.offsets, a.E, blockIdx.x / cols);
  if (blk.e < 0) return;
  const int mt = (min(blk.end - blk.row0, 16 * kMaxMT) + 15) / 16;  // the same for the whole workgroup
  if (mt == 1) {
    RowsBody<XT, FMT, GPB, 1, W13>(a, blk, col_wg, abuf, xsum).run(col_wg);
  } else if (mt == 2) {
    RowsBody<XT, FMT, GPB, 2, W13>(a, blk, col_wg, abuf, xsum).run(col_wg);
  } else if constexpr (kMaxMT > 2) {
    RowsBody<XT, FMT, GPB, 3, W13>(a, blk, col_wg, abuf, xsum).run(col_wg);
  }
}

// Launch over every row block (an upper bound of their number is known on the
// host; workgroups past the last exit at once).
template <typename XT, bool W13>
inline hipError_t launch_rows_of(const Shape& s, const Q4& q, const Q4Rows& a, hipStream_t st) {
  constexpr int kRows = sizeof(XT) == 2 ? 48 : 32;
  const long long blocks = s.R() / kRows + (s.R() < s.E ? s.R() : s.E);
  const dim3 grid((unsigned)(blocks * ((a.tiles + kQrColTiles<XT> - 1) / kQrColTiles<XT>))), block(kQrWaves * 64);
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
