// How the router's gradient is cut (csrc/pw_internal.h): a workspace for T
// tokens holds the shares of every call of up to T, and is not much larger than
// the largest of them needs.  Host code only.
#include <stdio.h>
#include <stdlib.h>

#include "pw_internal.h"

int main() {
  const int H[] = {32, 224, 512, 544, 1024, 1056, 2048, 4064, 4096, 7168, 8192, 16384};
  const int E[] = {1, 2, 8, 33, 60, 128, 157, 256};
  const int k[] = {1, 2, 3, 4, 8, 64};
  for (int h : H)
    for (int e : E)
      for (int kk : k) {
        if (kk > e) continue;
        size_t most = 0, last = 0;
        for (int64_t T = 0; T <= (1 << 20); T += T < 3000 ? 1 : T / 97) {
          const pw::RouterGradPlan p = pw::router_grad_plan(h, e, kk, T);
          const size_t share = sizeof(float) * (size_t)e * h, used = p.splits > 1 ? p.splits * share : 0;
          if (used > most) most = used;
          const bool covered = p.splits * p.split_slots >= T * kk;
          // the stretches are whole in slots, so a call may have fewer than the rule would allow
          if (p.bytes < most || p.bytes < last || p.bytes > 2 * most + share + 256 || !covered) {
            printf("H %d E %d k %d T %lld: %zu bytes, %d stretches use %zu, the largest so far %zu\n", h, e, kk,
                   (long long)T, p.bytes, p.splits, used, most);
            return 1;
          }
          last = p.bytes;
        }
      }
  printf("ok\n");
  return 0;
}
