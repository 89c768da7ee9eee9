// Tile sizes of the tiled products (tile_gemm.h), and which one a launch takes
// (host arithmetic only).
#pragma once

#include <stdint.h>

namespace moe {
namespace tile {

// What a tile size costs: ns per 128 bytes of k with 1, 2, ... workgroups on
// every CU (as many as LDS holds), measured at K = 4096 (bf16, average of a
// product with both operands k-contiguous and one with both k-rows) and 2048
// (fp32), and ns a tile beside that.
struct TileCost {
  int bm, bn, resident;
  int step[3];
};
template <class E>
struct TileCosts;
template <>
struct TileCosts<uint16_t> {
  static constexpr int COUNT = 6;
  static constexpr TileCost C[COUNT] = {{32, 64, 3, {185, 290, 420}}, {64, 64, 2, {230, 400, 0}}, {64, 128, 1, {340, 0, 0}},
                                        {128, 128, 1, {490, 0, 0}},   {128, 256, 1, {880, 0, 0}}, {256, 256, 1, {1630, 0, 0}}};
};
// No 64 x 128: its 1000 ns are always more than the 980 of two 64 x 64 that share
// a CU in its place.
template <>
struct TileCosts<float> {
  static constexpr int COUNT = 3;
  static constexpr TileCost C[COUNT] = {{32, 64, 3, {300, 540, 770}}, {64, 64, 2, {520, 980, 0}}, {128, 128, 1, {1890, 0, 0}}};
};

inline long long tile_ns(const TileCost& c, long long steps, int resident) {
  return steps * c.step[resident - 1] + 2200 + c.bm * c.bn / 8;
}
constexpr int kCus = 256;
template <class E, class F>
int cheapest(F ns) {
  int best = 0;
  for (int i = 1; i < TileCosts<E>::COUNT; ++i)
    if (ns(TileCosts<E>::C[i]) < ns(TileCosts<E>::C[best])) best = i;
  return best;
}
inline long long tiles_of(const TileCost& c, long long M, long long N) {
  return ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
}
template <class E>
long long steps_of(long long K) {
  return (K * (long long)sizeof(E) + 127) / 128;
}

// Estimated ns of an M x N product: whole rounds of `resident` tiles a CU, and
// what is left.
inline long long product_ns(const TileCost& c, long long M, long long N, long long steps) {
  const long long a_cu = (tiles_of(c, M, N) + kCus - 1) / kCus;
  const int left = (int)(a_cu % c.resident);
  return a_cu / c.resident * tile_ns(c, steps, c.resident) + (left ? tile_ns(c, steps, left) : 0);
}
// Index of the tile size for an M x N product over K.
template <class E>
int product_tile(long long M, long long N, long long K) {
  return cheapest<E>([&](const TileCost& c) { return product_ns(c, M, N, steps_of<E>(K)); });
}

// Estimated ns until `n1` tiles of `a` ns and behind them `n2` of `b` ns are
// done, every tile going to the place that is free first.
inline long long makespan(long long n1, long long a, long long n2, long long b, long long places) {
  // the places that hold one tile of the first kind more, and the others
  const long long extra = n1 % places;
  long long t_extra = (n1 / places + 1) * a, t = n1 / places * a;
  while (n2 > 0) {
    const bool e = extra > 0 && t_extra <= t;
    (e ? t_extra : t) += b;
    n2 -= e ? extra : places - extra;
  }
  return extra > 0 && t_extra > t ? t_extra : t;
}
// Index of the tile size for two products of one launch, the one with the
// longer sums first.  M == 0: that one is not wanted.
struct Extent {
  long long M, N, K;
};
template <class E>
int pair_tile(const Extent& x, const Extent& w) {
  return cheapest<E>([&](const TileCost& c) {
    const long long nx = tiles_of(c, x.M, x.N), nw = tiles_of(c, w.M, w.N), a_cu = (nx + nw + kCus - 1) / kCus;
    const int resident = a_cu < 1 ? 1 : a_cu < c.resident ? (int)a_cu : c.resident;
    const long long ns_x = tile_ns(c, steps_of<E>(x.K), resident), ns_w = tile_ns(c, steps_of<E>(w.K), resident);
    return w.K > x.K ? makespan(nw, ns_w, nx, ns_x, kCus * resident) : makespan(nx, ns_x, nw, ns_w, kCus * resident);
  });
}

}  // namespace tile
}  // namespace moe
