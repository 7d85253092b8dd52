// How many parts a cut tile of the expert products has (csrc/pw_internal.h): the
// number that saves most by the rule's three times, the fewest where several do,
// whatever the compiler fuses.  Host code only.
#include <stdio.h>

#include "pw_internal.h"

int main() {
  long ties = 0;
  for (unsigned BM : {32u, 64u, 128u, 256u}) {
    const unsigned together = pw::product_blocks((int)BM);
    if (pw::product_parts(BM, 0, 100, together) != 1) return 1;
    for (unsigned rest = 1; rest < together; ++rest)
      for (unsigned steps = 1; steps <= 4096; steps += steps < 700 ? 1 : 97) {
        // tenths of a us, times 256
        auto saved = [&](unsigned p) {
          return 13LL * 256 * (steps - (steps + p - 1) / p) - 1LL * BM * rest * p;
        };
        const unsigned parts = pw::product_parts(BM, rest, steps, together);
        bool right = parts >= 1 && parts <= (unsigned)pw::kProdParts && (parts == 1 || (rest * parts <= together && 2 * parts <= steps));
        if (parts > 1) right = right && saved(parts) > 50 * 256;
        for (unsigned p = 2; p <= 16 && 2 * p <= steps && rest * p <= together; ++p) {
          const long long least = parts > 1 ? saved(parts) : 50 * 256;
          right = right && saved(p) <= least && (p >= parts || saved(p) < least);
          ties += p != parts && saved(p) == least;
        }
        if (!right) {
          printf("BM %u rest %u steps %u: %u parts\n", BM, rest, steps, parts);
          return 1;
        }
      }
  }
  if (!ties) return 2;
  printf("ok\n");
  return 0;
}
