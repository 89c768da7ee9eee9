// Tile sizes that the library's launches choose (csrc/tile_choice.h), for
// tests: reads one question a line, answers with the tile's rows and columns.
//   sizes TYPE                         all tile sizes of the type
//   product TYPE M N K                 an M x N product over K
//   pair TYPE M N K  M N K             two products of one launch (rows, then a weight's gradient)
#include <stdio.h>
#include <string.h>

#include "tile_choice.h"

using namespace moe::tile;

template <class E>
static int answer(const char* what) {
  long long a[6];
  if (strcmp(what, "sizes") == 0) {
    for (int i = 0; i < TileCosts<E>::COUNT; ++i) printf("%d %d ", TileCosts<E>::C[i].bm, TileCosts<E>::C[i].bn);
    printf("\n");
    return 0;
  }
  const int n = strcmp(what, "product") == 0 ? 3 : strcmp(what, "pair") == 0 ? 6 : 0;
  for (int i = 0; i < n; ++i)
    if (scanf("%lld", &a[i]) != 1) return 1;
  if (n == 0) return 1;
  const int i = n == 3 ? product_tile<E>(a[0], a[1], a[2]) : pair_tile<E>({a[0], a[1], a[2]}, {a[3], a[4], a[5]});
  printf("%d %d\n", TileCosts<E>::C[i].bm, TileCosts<E>::C[i].bn);
  return 0;
}

int main() {
  char what[16], type[16];
  while (scanf("%15s %15s", what, type) == 2)
    if (strcmp(type, "bf16") == 0 ? answer<uint16_t>(what) : answer<float>(what)) return 1;
  return 0;
}
