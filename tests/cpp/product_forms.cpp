// Which form of the expert products a call takes (csrc/pw_internal.h).  Host code
// only.  Every line of the input is
//   product KIND Z8 E S N K RAGGED [rows of every expert]   KIND: 0 product, 1 gated, 2 back, 3 gated, back
//   outer E S M N
// and is answered by "few", "ROWS whole" or "ROWS cut" (rows of a tile; whether
// tiles of this call are cut along the reduction), or by "ROWSxCOLUMNS PARTS".
#include <stdio.h>
#include <string.h>

#include "pw_internal.h"

int main() {
  char what[16];
  while (scanf("%15s", what) == 1) {
    if (!strcmp(what, "outer")) {
      int E, S, M, N;
      if (scanf("%d %d %d %d", &E, &S, &M, &N) != 4) return 1;
      const bool small = pw::outer_is_small(E, M, N);
      printf("%s %d\n", small ? "128x128" : pw::outer_is_short(E, S) ? "256x128" : "256x256", pw::outer_parts(E, S, M, N));
      continue;
    }
    int kind, z8, E, S, N, K, ragged;
    if (scanf("%d %d %d %d %d %d %d", &kind, &z8, &E, &S, &N, &K, &ragged) != 7) return 1;
    const int NT = pw::product_col_tiles(kind, N), BM = pw::product_rows(E, S, NT);
    int64_t row_tiles = 0;
    for (int e = 0; e < E; ++e) {
      int n = S;
      if (ragged && scanf("%d", &n) != 1) return 1;
      row_tiles += (n + BM - 1) / BM;
    }
    const bool forward = kind == pw::kProductAct || kind == pw::kProductGate;
    const int64_t matrix = (int64_t)N * K * (kind == pw::kProductGate ? 2 : 1);
    if (forward && !z8 && pw::few_rows_for(E, S, matrix)) {
      puts("few");
      continue;
    }
    const int64_t bound = pw::product_row_tiles(ragged != 0, E, S, BM) * NT;
    const int steps = (K + pw::kProdK - 1) / pw::kProdK;
    const unsigned together = pw::product_blocks(BM), rest = (unsigned)(row_tiles * NT % together);
    const bool scratch = !forward || !pw::few_rows_for(E, S, matrix);
    const bool cut = scratch && pw::product_is_cut(ragged != 0, bound, steps, BM) && pw::product_parts(BM, rest, steps, together) > 1;
    printf("%d %s\n", BM, cut ? "cut" : "whole");
  }
  return 0;
}
