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

DF2_HD inline UnitKeys paged_unit_keys(const PagedShape& s, int n, int len, int qt) {
  const int row1 = (qt + 1) * s.rows < n * s.group ? (qt + 1) * s.rows : n * s.group;
  const int p0 = len - n + qt * s.rows / s.group, p1 = len - n + (row1 - 1) / s.group;
  UnitKeys u;
  u.hi = s.causal == 1 ? p1 + 1 : len;
  if (u.hi < 0) u.hi = 0;
  u.lo = s.window > 0 && p0 - s.window + 1 > 0 ? p0 - s.window + 1 : 0;
  if (u.lo > u.hi) u.lo = u.hi;
  u.t0 = u.lo / s.bn;
  u.nt = (u.hi + s.bn - 1) / s.bn - u.t0;
  if (u.nt < 1) u.nt = 1;
  return u;
}

// Tiles of one KV head of a request.
DF2_HD inline long long paged_head_tiles(const PagedShape& s, int n, int len) {
  long long t = 0;
  const int nq = paged_row_tiles(s, n);
  for (int qt = 0; qt < nq; ++qt) t += paged_unit_keys(s, n, len, qt).nt;
  return t;
}

// First tile of CTA c's run.
DF2_HD inline long long paged_run_begin(long long c, long long C, long long T) { return c * T / C; }

// Whether the run [t0, t1) has a tile of the request whose tiles are [first, next).
DF2_HD inline bool paged_in_run(long long first, long long next, long long t0, long long t1) {
  return first < next && first < t1 && next > t0;
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
  // row of the request, its new tokens), or -1; whether one of the CTA's waits gave up
  int* desc;
  unsigned* count;   // [CTAs] partials of that unit that have come (zero between calls)
  int ctas;
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

}  // namespace df2
