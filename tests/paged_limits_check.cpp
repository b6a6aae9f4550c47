// The attention's schedule (paged.h) at the longest caches and the most rows, for the compiler's overflow checks: host
// code, no GPU.  Prints "ok <cases>" or the first difference.
#include <cstdio>

#include "paged.h"

using namespace df2;

int main() {
  long long cases = 0;
  for (int len : {kPagedMaxLen, kPagedMaxLen - 1, kPagedMaxLen - 127})
    for (int n : {1, 33, 100000, len})
      for (int rows : {16, 32, 256})
        for (int bn : {64, 128})
          for (int causal = 0; causal < 3; ++causal)
            for (int w : {0, 1, 4096, 1 << 30})
              for (int group : {1, 4, 64}) {
                if (static_cast<long long>(n) * group > kPagedMaxRows) continue;
                const PagedShape s{group, rows, bn, causal, w};
                const int nq = paged_row_tiles(s, n);
                if (static_cast<long long>(nq) * rows < static_cast<long long>(n) * group) return std::printf("rows %d %d\n", n, group), 1;
                for (int qt : {0, nq / 2, nq - 1}) {
                  const UnitKeys u = paged_unit_keys(s, n, len, qt);
                  if (u.lo < 0 || u.hi > len || u.lo > u.hi || u.nt < 1 || u.t0 < 0 ||
                      static_cast<long long>(u.t0 + u.nt) * bn < u.hi || static_cast<long long>(u.t0 + u.nt) * bn > 0x7FFFFFFFll + 1)
                    return std::printf("unit %d %d %d\n", len, n, qt), 1;
                  ++cases;
                }
              }
  std::printf("ok %lld\n", cases);
  return 0;
}
