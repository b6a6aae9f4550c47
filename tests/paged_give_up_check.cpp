// What a prefix's launch spoils when a wait of a CTA gives up (paged.h), against its tiles one by one: the groups with a tile in
// the CTA's run, and every row of those groups once.  Host code, no GPU.  Prints "ok <cases>" or the first difference.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "paged.h"

using namespace df2;

int main() {
  long long cases = 0;
  std::srand(11);
  for (int trial = 0; trial < 300; ++trial) {
    const int groups = 1 + std::rand() % 6, n_kv = 1 + std::rand() % 3;
    PagedShape s = {};
    s.group = 1 + std::rand() % 5;
    s.rows = kChunkRows, s.bn = kChunkBn;
    const int heads = n_kv * s.group;
    std::vector<int> b0(groups), n(groups), len(groups);
    int tokens = 0;
    for (int g = 0; g < groups; ++g) {
      b0[g] = tokens;
      n[g] = std::rand() % 4 ? std::rand() % 300 : 0;  // (0: a group without a part in this launch)
      len[g] = 1 + std::rand() % 900;
      tokens += n[g] + std::rand() % 3;  // (rows of groups that take no part lie between)
    }
    std::vector<int> group_of;                       // of each tile
    std::vector<std::vector<int>> rows_of;           // the (token, head) rows of each tile's unit
    for (int g = 0; g < groups; ++g)
      for (int h = 0; n[g] > 0 && h < n_kv; ++h)
        for (int qt = 0; qt < paged_row_tiles(s, n[g]); ++qt) {
          std::vector<int> rows;
          for (int row = qt * s.rows; row < (qt + 1) * s.rows && row < n[g] * s.group; ++row)
            rows.push_back((b0[g] + row / s.group) * heads + h * s.group + row % s.group);
          for (int i = 0; i < paged_unit_keys(s, n[g], len[g], qt).nt; ++i) group_of.push_back(g), rows_of.push_back(rows);
        }
    const long long T = static_cast<long long>(group_of.size());
    auto tiles = [&](int g) { return n[g] > 0 ? n_kv * paged_head_tiles(s, n[g], len[g]) : 0ll; };
    for (long long ctas = 1; ctas <= 40; ctas += 1 + std::rand() % 7) {
      const long long C = T < ctas ? T : ctas;
      for (long long c = 0; c < ctas; ++c, ++cases) {
        std::vector<bool> found(groups, false);
        std::vector<int> spoiled(static_cast<size_t>(tokens) * heads, 0);
        paged_beside_run(groups, ctas, c, tiles, [&](int g, long long first, long long next, long long t0, long long t1) {
          if (!paged_in_run(first, next, t0, t1)) return;
          found[g] = true;
          for (int thread = 0; thread < 128; ++thread)
            paged_each_row(b0[g], n[g], heads, thread, 128, [&](int token, int head) { ++spoiled.at(token * heads + head); });
        });
        std::vector<bool> want(groups, false);
        std::vector<int> rows(spoiled.size(), 0);
        const long long t0 = c < C ? paged_run_begin(c, C, T) : 0, t1 = c < C ? paged_run_begin(c + 1, C, T) : 0;
        for (long long t = t0; t < t1; ++t) {
          want[group_of[t]] = true;
          for (int row : rows_of[t])
            if (!spoiled.at(row)) {
              std::printf("trial %d, run %lld of %lld: row %d keeps what it held\n", trial, c, C, row);
              return 1;
            }
        }
        for (int g = 0; g < groups; ++g)
          for (int i = 0; i < n[g] * heads; ++i) rows[b0[g] * heads + i] = want[g];
        if (found != want || spoiled != rows) {
          std::printf("trial %d, run %lld of %lld\n", trial, c, C);
          return 1;
        }
      }
    }
  }
  std::printf("ok %lld\n", cases);
  return 0;
}
