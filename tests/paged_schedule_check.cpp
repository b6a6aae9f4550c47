// The attention's schedule (paged.h) against brute force, and the bounds checks of the
// paged cache: host code, no GPU.  Prints "ok <cases>" or the first difference.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "paged.h"

using namespace df2;

static int fail(const char* what, int a, int b, int c, int d) {
  std::printf("%s: %d %d %d %d\n", what, a, b, c, d);
  return 1;
}

int main() {
  long long cases = 0;
  const int ns[] = {0, 1, 2, 7, 8, 33, 64, 65, 130}, lens[] = {0, 1, 5, 63, 64, 65, 129, 200, 517};
  const int groups[] = {1, 3, 4, 8, 64}, rowss[] = {16, 32, 64, 128, 256}, bns[] = {64, 128}, windows[] = {0, 1, 40, 2048};
  for (int n : ns)
    for (int len : lens)
      for (int g : groups)
        for (int rows : rowss)
          for (int bn : bns)
            for (int causal = 0; causal < 3; ++causal)
              for (int w : windows) {
                PagedShape s{g, rows, bn, causal, w};
                const int nq = paged_row_tiles(s, n);
                if (nq * rows < n * g || (nq - 1) * rows >= n * g + (n == 0)) return fail("row tiles", n, g, rows, nq);
                long long total = 0;
                for (int qt = 0; qt < nq; ++qt) {
                  const UnitKeys u = paged_unit_keys(s, n, len, qt);
                  if (u.nt < 1 || u.lo < 0 || u.hi > len || u.lo > u.hi) return fail("range", n, len, qt, u.nt);
                  total += u.nt;
                  for (int row = qt * rows; row < (qt + 1) * rows && row < n * g; ++row) {
                    const int p = len - n + row / g;
                    for (int j = 0; j < len; ++j) {
                      const bool see = (causal != 1 || j <= p) && (w == 0 || p - j < w);
                      if (see && (j < u.lo || j >= u.hi || j / bn < u.t0 || j / bn >= u.t0 + u.nt))
                        return fail("a visible key outside the unit", n, len, row, j);
                    }
                  }
                  ++cases;
                }
                if (total != paged_head_tiles(s, n, len)) return fail("tiles", n, len, g, rows);
              }
  // runs: every tile in exactly one, none empty when there are no more CTAs than tiles, and the CTA of a
  // tile as the combine computes it
  for (long long T : {1ll, 2ll, 7ll, 303ll, 304ll, 305ll, 100001ll})
    for (long long C = 1; C <= 304 && C <= T; ++C) {
      long long t = 0;
      for (long long c = 0; c < C; ++c) {
        const long long b = paged_run_begin(c, C, T), e = paged_run_begin(c + 1, C, T);
        if (b != t || e <= b) return fail("run", (int)T, (int)C, (int)c, (int)b);
        for (long long x : {b, e - 1})
          if (((x + 1) * C - 1) / T != c) return fail("tile's CTA", (int)T, (int)C, (int)c, (int)x);
        t = e;
        ++cases;
      }
      if (t != T) return fail("runs' end", (int)T, (int)C, (int)t, 0);
    }
  // offsets past 32 bits, and ids outside the pool
  PagedCache c{};
  c.n_pages = 5000;
  c.page_stride = 1ll << 22;
  c.token_stride = 1 << 10;
  c.head_stride = 128;
  c.s_page_stride = 1 << 15;
  c.s_token_stride = 8;
  c.s_head_stride = 1;
  long long off = -7, soff = -7;
  if (!paged_row(c, 4999, 63, 7, &off, &soff) || off != 4999ll * (1ll << 22) + 63 * 1024 + 7 * 128 ||
      soff != 4999ll * 32768 + 63 * 8 + 7)
    return fail("offset", 0, 0, 0, 0);
  off = soff = -7;
  for (int page : {-1, 5000, 2147483647, -2147483647 - 1})
    if (paged_row(c, page, 0, 0, &off, &soff) || off != -7 || soff != -7) return fail("page id", page, 0, 0, 0);
  PagedReq q{};
  q.n_tokens = 100;
  q.max_new = 40;
  q.max_len = 1000;
  if (!paged_request_ok(q, 0, 40, 1000) || !paged_request_ok(q, 100, 100, 0)) return fail("good request", 0, 0, 0, 0);
  const int bad[][3] = {{-1, 3, 10}, {5, 4, 10}, {90, 101, 50}, {0, 41, 50}, {0, 3, 1001}, {0, 3, -1}};
  for (auto& b : bad)
    if (paged_request_ok(q, b[0], b[1], b[2])) return fail("bad request", b[0], b[1], b[2], 0);
  std::printf("ok %lld\n", cases);
  return 0;
}
