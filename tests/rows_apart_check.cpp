// Whether rows overlap (paged_api.h), against their channels one by one: host code, no GPU.  Prints "ok <cases>" or the first
// difference.
#include <cstdio>
#include <set>

#include "paged_api.h"

using namespace df2;

int main() {
  long long cases = 0, apart = 0;
  for (int dim = 1; dim <= 3; ++dim)
    for (int tokens = 1; tokens <= 5; ++tokens)
      for (int heads = 1; heads <= 5; ++heads)
        for (int t = -13; t <= 13; ++t)
          for (int h = -13; h <= 13; ++h, ++cases) {
            std::set<int> seen;
            bool want = true;
            for (int i = 0; i < tokens; ++i)
              for (int j = 0; j < heads; ++j)
                for (int c = 0; c < dim; ++c) want &= seen.insert(i * t + j * h + c).second;
            dflash2_rows r = {};
            r.token_stride = t, r.head_stride = h;
            if (rows_apart(r, tokens, heads, dim) != want) {
              std::printf("%d tokens %d apart, %d heads %d apart, of %d\n", tokens, t, heads, h, dim);
              return 1;
            }
            apart += want;
          }
  std::printf("ok %lld, %lld of them apart\n", cases, apart);
  return 0;
}
