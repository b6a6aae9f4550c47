// Which requests a CTA's run of tiles touches (paged.h), against the tiles one by one: host code, no GPU.  Prints
// "ok <cases>" or the first difference.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "paged.h"

using namespace df2;

int main() {
  long long cases = 0;
  std::srand(5);
  for (int trial = 0; trial < 400; ++trial) {
    const int n = 1 + std::rand() % 12;
    std::vector<long long> pre(n + 1, 0);
    std::vector<int> of;  // the request of each tile
    for (int r = 0; r < n; ++r) {
      const int tiles = std::rand() % 3 ? std::rand() % 9 : 0;
      pre[r + 1] = pre[r] + tiles;
      of.insert(of.end(), tiles, r);
    }
    const long long T = pre[n];
    for (long long C = 1; C <= T && C <= 20; ++C)
      for (long long c = 0; c < C; ++c) {
        const long long t0 = paged_run_begin(c, C, T), t1 = paged_run_begin(c + 1, C, T);
        std::vector<bool> want(n, false);
        for (long long t = t0; t < t1; ++t) want[of[t]] = true;
        for (int r = 0; r < n; ++r, ++cases)
          if (paged_in_run(pre[r], pre[r + 1], t0, t1) != want[r]) {
            std::printf("trial %d, run %lld of %lld, request %d\n", trial, c, C, r);
            return 1;
          }
      }
  }
  std::printf("ok %lld\n", cases);
  return 0;
}
