// The paged K/V cache and the attention over it: argument blocks, launch interfaces,
// and the schedule of the attention's work (shared by host checks and kernels).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace df2 {

enum { kKvBf16 = 0, kKvF16 = 1, kKvInt8 = 2, kKvE4m3 = 3 };
enum { kTBf16 = 0, kTF16 = 1, kTF32 = 2 };

// One layer's pools and the call's requests, as the kernels take them.
struct PagedCache {
  char* k;
  char* v;
  float* k_scale;
  float* v_scale;
  const int32_t* table;
  long long page_stride, token_stride, head_stride;        // elements
  long long s_page_stride, s_token_stride, s_head_stride;  // scales
  long long table_stride;
  int n_pages, max_pages, page_size, n_kv;
};

struct PagedReq {
  const int32_t* begin;   // [n_req + 1]
  const int32_t* kv_len;  // [n_req]
  int32_t* status;        // [n_req] or null
  int n_req, n_tokens;
  int max_new, max_len;   // bounds a request must keep
};

struct PagedRows {
  char* p;
  long long token_stride, head_stride;  // elements
  int type;
};

// Element offset of (page, row of the page, KV head) in a pool with these strides; false, and no
// offset, for a page id outside the pool.
DF2_HD inline bool paged_row(const PagedCache& c, int page, int row, int h, long long* off, long long* soff) {
  if (page < 0 || page >= c.n_pages) return false;
  *off = page * c.page_stride + row * c.token_stride + h * c.head_stride;
  *soff = page * c.s_page_stride + row * c.s_token_stride + h * c.s_head_stride;
  return true;
}

// In the place of an offset where there is no row.  (Strides may be negative, so offsets may; this one no pool reaches.)
constexpr long long kNoRow = -0x7FFFFFFFFFFFFFFFll - 1;

// Whether a request's rows [b0, b1) and cache length are within the call's bounds.
DF2_HD inline bool paged_request_ok(const PagedReq& q, int b0, int b1, int len) {
  return b0 >= 0 && b1 >= b0 && b1 <= q.n_tokens && b1 - b0 <= q.max_new && len >= 0 && len <= q.max_len;
}

struct PagedMoveArgs {
  PagedCache c;
  PagedReq rq;
  PagedRows k, v;
};
cudaError_t launch_paged_write(const PagedMoveArgs& a, int head_dim, int fmt, cudaStream_t st);
cudaError_t launch_paged_read(const PagedMoveArgs& a, int head_dim, int fmt, cudaStream_t st);

// Longest cache of a request, and most rows (new tokens x group) of one: rounded up to a tile they stay in 32 bits.
constexpr int kPagedMaxLen = 0x7FFFFFFF - 511, kPagedMaxRows = 0x7FFFFFFF - 511;

// ------------------------------------------------------------------ attention schedule
// The rows of a request are its (token, query head of one KV head) pairs, token-major:
// row = i * group + g.  A unit is (request, KV head, tile of `rows` rows); it reads the
// union of its rows' visible keys in tiles of `bn` keys (aligned to bn).  Units are
// ordered by request, then KV head, then row tile, and the launch's tiles, numbered
// through, are dealt to the CTAs in contiguous runs: CTA c of C takes
// [floor(c T / C), floor((c + 1) T / C)).  A unit cut by a run's end leaves partial
// results that the combine kernel joins in CTA order.
struct PagedShape {
  int group, rows, bn;
  int causal;  // 0: all keys, 1: keys up to the token's position, 2: tree mask (all keys, then bits)
  int window;
};

struct UnitKeys {
  int lo, hi;  // keys some row sees: [lo, hi)
  int t0, nt;  // tiles t0 .. t0 + nt - 1 (at least one: a unit that sees nothing still writes its rows)
};

DF2_HD inline int paged_row_tiles(const PagedShape& s, int n) { return (n * s.group + s.rows - 1) / s.rows; }

// from: keys below it are not this unit's.
DF2_HD inline UnitKeys paged_unit_keys(const PagedShape& s, int n, int len, int qt, int from = 0) {
  const int row1 = (qt + 1) * s.rows < n * s.group ? (qt + 1) * s.rows : n * s.group;
  const int p0 = len - n + qt * s.rows / s.group, p1 = len - n + (row1 - 1) / s.group;
  UnitKeys u;
  u.hi = s.causal == 1 ? p1 + 1 : len;
  if (u.hi < 0) u.hi = 0;
  u.lo = s.window > 0 && p0 - s.window + 1 > from ? p0 - s.window + 1 : from;
  if (u.lo > u.hi) u.lo = u.hi;
  u.t0 = u.lo / s.bn;
  u.nt = (u.hi + s.bn - 1) / s.bn - u.t0;
  if (u.nt < 1) u.nt = 1;
  return u;
}

// Tiles of one KV head of a request.
DF2_HD inline long long paged_head_tiles(const PagedShape& s, int n, int len, int from = 0) {
  long long t = 0;
  const int nq = paged_row_tiles(s, n);
  for (int qt = 0; qt < nq; ++qt) t += paged_unit_keys(s, n, len, qt, from).nt;
  return t;
}

// First tile of CTA c's run.
DF2_HD inline long long paged_run_begin(long long c, long long C, long long T) { return c * T / C; }

// Whether the run [t0, t1) has a tile of the request whose tiles are [first, next).
DF2_HD inline bool paged_in_run(long long first, long long next, long long t0, long long t1) {
  return first < next && first < t1 && next > t0;
}

// Calls see(r, first, next, t0, t1) for each request, whose tiles are [first, next), beside CTA c's run [t0, t1) of a launch of
// `ctas` CTAs; tiles(r): request r's tiles.
#ifdef __CUDACC__
#pragma nv_exec_check_disable
#endif
template <typename Tiles, typename See>
DF2_HD inline void paged_beside_run(int n_req, long long ctas, long long c, const Tiles& tiles, const See& see) {
  long long T = 0, first = 0;
  for (int r = 0; r < n_req; ++r) T += tiles(r);
  const long long C = T < ctas ? T : ctas;
  if (c >= C) return;
  for (int r = 0; r < n_req; ++r) {
    const long long next = first + tiles(r);
    see(r, first, next, paged_run_begin(c, C, T), paged_run_begin(c + 1, C, T));
    first = next;
  }
}

// Every `step`th of the rows (token, query head) of tokens b0 .. b0 + n - 1, from the `first` on.
#ifdef __CUDACC__
#pragma nv_exec_check_disable
#endif
template <typename Row>
DF2_HD inline void paged_each_row(int b0, int n, int heads, int first, int step, const Row& row) {
  const long long rows = static_cast<long long>(n) * heads;
  for (long long i = first; i < rows; i += step) row(b0 + static_cast<int>(i / heads), static_cast<int>(i % heads));
}

// Requests in groups that share a prefix: two launches.  In the first the call's "requests" are the groups of more than one: their
// rows see all of the prefix, and each row's result (outputs not divided by the sum, and maximum and sum) goes to the
// workspace.  In the second they are the requests, with the keys behind the prefix, and what they write has the prefix's
// part in it.  Or (`apart`) one launch of the requests, each with all its keys.
struct PagedGroups {
  const int32_t* begin;   // [n_groups + 1]
  const int32_t* prefix;  // [n_groups]
  int n_groups, n_req;
  int max_group, max_prefix;
  int first, second;      // the first launch, or a second after one
  int apart;              // (before the launch: the caller's choice)
  float* joint;           // [n_tokens * query heads][head_dim], then as many (maximum, sum)
};

enum { kSharedAuto = 0, kSharedTogether = 1, kSharedApart = 2 };
// Apart, the requests behind a group's first one read its prefix again, mostly from L2; together, there is a launch more, a
// join of its partials, and a part to fetch for every row.  Bytes read again where the two meet: for units of 16 rows, twice
// that for wider ones.  Measured (us; together / apart), 8 KV heads of 128, 4 KB a position in bf16 and 2.1 in e4m3, single tokens: bf16
// 4 requests over 8192 positions 32 / 29, 8 over 4096 29 / 29, 16 over 1024 24 / 21, over 2048 27 / 29, 64 over 512 34 / 33, over 1024
// 35 / 50; e4m3 4 over 16384 38 / 37, 16 over 2048 31 / 26, over 4096 33 / 38, 64 over 512 41 / 36, over 1024 42 / 45.  Blocks of 8:
// bf16 16 over 2048 42 / 35, over 4096 51 / 56, 64 over 1024 64 / 64; e4m3 16 over 4096 60 / 53, over 8192 70 / 88, 64 over 1024
// 80 / 66, over 2048 88 / 99.
// Other shapes go by the same border, which is then off on either side (us, together / apart, MiB read again; states in turn).  One KV
// head of 128, bf16: tokens 16 over 16384 (120) 36 / 28, 64 over 4096 (126) 28 / 30; blocks 16 over 16384 (120) 48 / 35, 64 over 4096 (126)
// 35 / 36.  Eight of 64: tokens 16 over 4096 (120) 22 / 37, e4m3 (64) 25 / 32; blocks 16 over 4096 (120) 34 / 41, 64 over 1024 (126) 50 / 47.
// Above 32 rows a unit, where products count and not bytes: trees of 33 nodes bf16 16 over 4096 (240) 93 / 88, 64 over 1024 (252) 154 /
// 122, over 4096 (1008) 231 / 280, e4m3 16 over 4096 (124) 100 / 118; chunks of 128 tokens bf16 16 over 4096 (240) 211 / 173, 64 over 1024
// (252) 366 / 250; of 301 tokens 8 over 16384 (448) 551 / 604.
constexpr long long kApartBytes = 100ll << 20;

// Whether group g's requests [g0, g1) follow those of the group before and, the last's, end at the last request.  (Where one
// does not, the whole call is refused: all of `begin` is trusted after that.)
DF2_HD inline bool paged_group_in_order(const PagedGroups& s, int g, int g0, int g1) {
  return g0 <= g1 && (g > 0 || g0 == 0) && (g < s.n_groups - 1 || g1 == s.n_req);
}
// Whether a group's prefix and rows [b0, b1) are within the call's bounds.
DF2_HD inline bool paged_group_ok(const PagedGroups& s, const PagedReq& q, int prefix, int b0, int b1) {
  return prefix >= 0 && prefix <= s.max_prefix && b0 >= 0 && b1 >= b0 && b1 <= q.n_tokens && b1 - b0 <= s.max_group;
}

struct PagedAttnArgs {
  PagedCache c;
  PagedReq rq;
  PagedShape s;
  PagedRows q, out;
  const unsigned long long* tree;
  float* lse;
  float scale_log2;  // score scale * log2(e)
  float* part;       // partial results: slots of rows * head_dim outputs, then rows * (max, sum)
  // [CTAs][8]: the cut unit that begins in CTA c's run (request, KV head, row tile, last CTA and first slot, first
  // row of the request, its new tokens), or -1; whether one of the CTA's waits gave up; with shared prefixes, whether
  // the unit's rows have a part in the workspace
  int* desc;
  unsigned* count;   // [CTAs] partials of that unit that have come (zero between calls)
  int ctas;
  PagedGroups g;     // with shared prefixes
};

// Rows of one unit of the kernel for few rows.
inline int paged_rows(int max_new, int group) { return static_cast<long long>(max_new) * group <= 16 ? 16 : 32; }
constexpr int kPagedMaxCtasPerSm = 2;
// The kernel for many rows: one CTA per SM, units of 256 rows against tiles of 128 keys.
constexpr int kChunkBn = 128;
constexpr int kChunkRows = 256;
// Most rows of a request for the kernel for few rows.  Above, one unit of the other reads the keys once where this one
// would read them again for every 32 rows.  Measured (us; few rows / many; bf16, int8, e4m3), 16 requests over 8192
// positions of 8 heads of 128: 32 rows 108 / 123, 105 / 147, 92 / 165; 64 rows 196 / 126, 187 / 150, 161 / 168.  Heads of
// 64: 78 / 102, 73 / 111, 67 / 114; 142 / 103, 128 / 113, 117 / 116.  One KV head of 128: 25 / 29, 27 / 36, 26 / 38;
// 36 / 34, 40 / 39, 38 / 41.  A window of 2048: 44 / 56, 43 / 57, 40 / 61; 64 / 59, 68 / 61, 62 / 65.  One request over
// 16384: 27 / 31, 30 / 34, 29 / 36; 36 / 31, 38 / 35, 36 / 38.
constexpr int kChunkMinRows = 32;
// Scratch of the partials: two slots for each CTA, of 32 rows (two CTAs per SM) or 256.
inline size_t paged_part_floats(int num_sms, int head_dim) {
  return static_cast<size_t>(num_sms) * 2 * kChunkRows * (head_dim + 2);
}
cudaError_t launch_paged_chunk(PagedAttnArgs& a, int head_dim, int fmt, int qtype, int num_sms, cudaStream_t st);
cudaError_t launch_paged_attention(PagedAttnArgs& a, int head_dim, int fmt, int qtype, int num_sms, cudaStream_t st);
// The same with a.g (both launches, one after the other); the first launch's kernel for many rows.
cudaError_t launch_shared_prefix(PagedAttnArgs& a, int head_dim, int fmt, int qtype, int num_sms, cudaStream_t st);
cudaError_t launch_shared_chunk(PagedAttnArgs& a, int head_dim, int fmt, int qtype, int num_sms, cudaStream_t st);
cudaError_t launch_shared_attention(PagedAttnArgs& a, int head_dim, int fmt, int qtype, int num_sms, cudaStream_t st);

}  // namespace df2
