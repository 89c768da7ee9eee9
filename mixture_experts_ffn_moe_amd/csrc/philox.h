// Counter-based random numbers of the dropout: Philox 4x32 with ten rounds
// (J. K. Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011).  One block of the counter (group,
// offset) under the key seed serves the eight elements 8 * group .. + 7, 16
// bits each, lowest first: a round is two 32 x 32 -> 64 multiplications, so
// ten rounds cost 2.5 of them an element, which a kernel bound by memory hides;
// 32 bits an element would cost twice that.
#pragma once

#include "moe_common.h"

namespace moe {

struct Dropout {
  const uint64_t* rng;  // device: seed, offset; null: no dropout
  uint32_t cut;         // an element is dropped where its 16 bits are below
  float scale;          // 65536 / (65536 - cut)
};

struct DropKey {
  uint32_t k0, k1, o0, o1;
};
__device__ __forceinline__ DropKey drop_key(const Dropout& d) {
  const uint64_t seed = d.rng[0], offset = d.rng[1];
  return DropKey{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}

__device__ __forceinline__ uint4 philox(uint64_t group, DropKey k) {
  uint32_t x0 = (uint32_t)group, x1 = (uint32_t)(group >> 32), x2 = k.o0, x3 = k.o1, k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
    x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
    x1 = (uint32_t)b;
    x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
    x3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(x0, x1, x2, x3);
}

// Element 8 * group + i after dropout, from the group's block: v scaled, or 0
// (whatever v is) where it is dropped.
__device__ __forceinline__ float dropped(float v, const uint4& b, int i, const Dropout& d) {
  const uint32_t w = i < 2 ? b.x : i < 4 ? b.y : i < 6 ? b.z : b.w;
  return ((i & 1) ? w >> 16 : w & 0xffffu) >= d.cut ? v * d.scale : 0.0f;
}

}  // namespace moe
