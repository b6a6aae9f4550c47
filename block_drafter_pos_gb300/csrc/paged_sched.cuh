// Device side of the attention's schedule: the launch's tile count, and a cursor over the
// tiles of one CTA's run (paged.h has the order).
#pragma once

#include "common.cuh"
#include "paged.h"

namespace df2 {

// New tokens and cache length of request r; n = 0 for a request that is out of bounds.
DF2_DEV bool paged_request(const PagedReq& q, int r, int& b0, int& n, int& len) {
  b0 = __ldg(q.begin + r);
  const int b1 = __ldg(q.begin + r + 1);
  len = __ldg(q.kv_len + r);
  n = b1 - b0;
  if (!paged_request_ok(q, b0, b1, len)) {
    n = 0;
    return false;
  }
  return true;
}

// Tiles before each request: pre[0 .. n_req] in shared memory; returns the launch's total.
// Called by every thread of the block.
template <int THREADS>
DF2_DEV long long paged_scan(const PagedAttnArgs& a, long long* pre, long long* tmp) {
  // tmp: THREADS / 32 + 1 words
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  long long base = 0;
  for (int r0 = 0; r0 < a.rq.n_req; r0 += THREADS) {
    const int r = r0 + threadIdx.x;
    long long w = 0;
    if (r < a.rq.n_req) {
      int b0, n, len;
      if (paged_request(a.rq, r, b0, n, len)) w = a.c.n_kv * paged_head_tiles(a.s, n, len);
      else if (blockIdx.x == 0 && a.rq.status) a.rq.status[r] = 1;  // DFLASH2_E_INVAL
    }
    long long x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) tmp[wid] = x;
    __syncthreads();
    long long before = base, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < wid) before += tmp[i];
      all += tmp[i];
    }
    if (r < a.rq.n_req) pre[r] = before + x - w;
    base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) pre[a.rq.n_req] = base;
  __syncthreads();
  return base;
}

// One tile at a time through a CTA's run [t, t1).
struct PagedCursor {
  long long t, t1;
  int r, h, qt;        // the unit
  int b0, n, len;      // its request
  UnitKeys u;
  int i;               // tile within the unit (0 .. u.nt - 1)
  long long unit_t;    // the unit's first tile in the launch's numbering

  DF2_DEV bool valid() const { return t < t1; }

  DF2_DEV void start(const PagedAttnArgs& a, const long long* pre, long long begin, long long end) {
    t = begin;
    t1 = end;
    if (t >= t1) return;
    int lo = 0, hi = a.rq.n_req;  // the last request with pre[r] <= t (requests without tiles are passed over)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= t) lo = mid;
      else hi = mid;
    }
    r = lo;
    paged_request(a.rq, r, b0, n, len);
    const long long head = (pre[r + 1] - pre[r]) / a.c.n_kv;
    long long off = t - pre[r];
    h = static_cast<int>(off / head);
    off -= h * head;
    qt = 0;
    u = paged_unit_keys(a.s, n, len, 0);
    while (off >= u.nt) {
      off -= u.nt;
      u = paged_unit_keys(a.s, n, len, ++qt);
    }
    i = static_cast<int>(off);
    unit_t = t - i;
  }

  // Tiles of the unit that are in this run, from the present one; skip() passes over them.
  DF2_DEV int piece() const {
    const long long left = t1 - t;
    return left < u.nt - i ? static_cast<int>(left) : u.nt - i;
  }
  DF2_DEV void skip(const PagedAttnArgs& a, int tiles) {
    t += tiles - 1;
    i += tiles - 1;
    next(a);
  }
  DF2_DEV bool unit_ends() const { return i == u.nt - 1; }

  DF2_DEV void next(const PagedAttnArgs& a) {
    ++t;
    if (++i < u.nt) return;
    if (t >= t1) return;
    i = 0;
    unit_t = t;
    if (++qt >= paged_row_tiles(a.s, n)) {
      qt = 0;
      if (++h >= a.c.n_kv) {
        h = 0;
        do {  // the run has another tile, so another request has rows
          ++r;
          paged_request(a.rq, r, b0, n, len);
        } while (n == 0 && r + 1 < a.rq.n_req);
      }
    }
    u = paged_unit_keys(a.s, n, len, qt);
  }
};

}  // namespace df2
