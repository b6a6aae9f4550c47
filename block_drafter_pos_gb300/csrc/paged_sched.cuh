// Device side of the attention's schedule: the launch's tile count, and a cursor over the
// tiles of one CTA's run (paged.h has the order).
#pragma once

#include "common.cuh"
#include "paged.h"
#include "paged_mma.cuh"

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

#ifndef DF2_SHARED_PREFIX
#define DF2_SHARED_PREFIX 0
#endif
// The attention's sources are compiled twice: for the requests of a call, and (SHARED) for groups of them with a
// shared prefix and for their own keys.  What a "request" of the schedule is:
struct PagedWork {
  int b0, n, len;  // its rows and keys; n = 0: nothing to do
  int from;        // its first key
  int row;         // its row of the page table
  int head, head_row;  // the row that holds the keys below `head`
};
template <bool SHARED>
DF2_DEV bool paged_work(const PagedAttnArgs& a, int r, PagedWork& w) {
  w.from = w.head = 0;
  w.row = w.head_row = r;
  if constexpr (!SHARED) {
    return paged_request(a.rq, r, w.b0, w.n, w.len);
  } else {
    int g = r;
    if (!a.g.first) {  // the last group that begins at or before the request
      int hi = a.g.n_groups;
      g = 0;
      while (hi - g > 1) {
        const int mid = (g + hi) >> 1;
        if (__ldg(a.g.begin + mid) <= r) g = mid;
        else hi = mid;
      }
    }
    const int g0 = __ldg(a.g.begin + g), g1 = __ldg(a.g.begin + g + 1), prefix = __ldg(a.g.prefix + g);
    w.b0 = w.n = w.len = 0;
    const int b0 = __ldg(a.rq.begin + g0), b1 = __ldg(a.rq.begin + g1);
    if (!paged_group_ok(a.g, a.rq, prefix, b0, b1)) return false;
    if (a.g.first) {
      if (prefix == 0 || g1 - g0 == 1) return true;  // (its rows have no part of a prefix)
      w.b0 = b0, w.n = b1 - b0, w.len = prefix, w.row = g0;
      return true;
    }
    PagedWork own;
    if (!paged_request(a.rq, r, own.b0, own.n, own.len) || own.b0 < b0 || own.b0 + own.n > b1 ||
        own.len - own.n < prefix)
      return false;
    w.b0 = own.b0, w.n = own.n, w.len = own.len;
    if (a.g.apart || g1 - g0 == 1) w.head = prefix, w.head_row = g0;
    else w.from = prefix;
    return true;
  }
}
// Notes an error for r: with groups, for all its requests.
template <bool SHARED>
DF2_DEV void paged_flag(const PagedAttnArgs& a, int r, int what) {
  if (!a.rq.status) return;
  if (SHARED && a.g.first) {
    for (int x = __ldg(a.g.begin + r); x < __ldg(a.g.begin + r + 1); ++x) a.rq.status[x] = what;
  } else {
    a.rq.status[r] = what;
  }
}

// Tiles before each request: pre[0 .. n_req] in shared memory; returns the launch's total.
// Called by every thread of the block.
template <int THREADS, bool SHARED>
DF2_DEV long long paged_scan(const PagedAttnArgs& a, long long* pre, long long* tmp) {
  // tmp: THREADS / 32 + 1 words
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  long long base = 0;
  bool groups_fine = true;
  if constexpr (SHARED) {
    bool bad = false;
    for (int g = threadIdx.x; g < a.g.n_groups; g += THREADS)
      bad |= !paged_group_in_order(a.g, g, __ldg(a.g.begin + g), __ldg(a.g.begin + g + 1));
    groups_fine = !__syncthreads_or(bad);
  }
  for (int r0 = 0; r0 < a.rq.n_req; r0 += THREADS) {
    const int r = r0 + threadIdx.x;
    long long w = 0;
    if (r < a.rq.n_req) {
      PagedWork k;
      if (groups_fine && paged_work<SHARED>(a, r, k)) w = k.n > 0 ? a.c.n_kv * paged_head_tiles(a.s, k.n, k.len, k.from) : 0;
      else if (blockIdx.x == 0 && a.rq.status && !(SHARED && a.g.first)) a.rq.status[r] = 1;  // DFLASH2_E_INVAL
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
template <bool SHARED>
struct PagedCursor {
  long long t, t1;
  int r, h, qt;        // the unit
  int b0, n, len;      // its request
  int from, row, head, head_row;  // (SHARED)
  UnitKeys u;
  int i;               // tile within the unit (0 .. u.nt - 1)
  long long unit_t;    // the unit's first tile in the launch's numbering

  DF2_DEV bool valid() const { return t < t1; }
  DF2_DEV int table_row(int key) const { return SHARED ? (key < head ? head_row : row) : r; }
  DF2_DEV int first_key() const { return SHARED ? from : 0; }
  DF2_DEV void request(const PagedAttnArgs& a) {
    if constexpr (SHARED) {
      PagedWork w;
      paged_work<true>(a, r, w);
      b0 = w.b0, n = w.n, len = w.len, from = w.from, row = w.row, head = w.head, head_row = w.head_row;
    } else {
      paged_request(a.rq, r, b0, n, len);
    }
  }

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
    request(a);
    const long long head = (pre[r + 1] - pre[r]) / a.c.n_kv;
    long long off = t - pre[r];
    h = static_cast<int>(off / head);
    off -= h * head;
    qt = 0;
    u = paged_unit_keys(a.s, n, len, 0, first_key());
    while (off >= u.nt) {
      off -= u.nt;
      u = paged_unit_keys(a.s, n, len, ++qt, first_key());
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
          request(a);
        } while (n == 0 && r + 1 < a.rq.n_req);
      }
    }
    u = paged_unit_keys(a.s, n, len, qt, first_key());
  }
};

// Row (token, query head) of the workspace: where its outputs are, and its (maximum, sum).
template <int D>
DF2_DEV float* joint_row(const PagedAttnArgs& a, int token, int head) {
  return a.g.joint + (static_cast<long long>(token) * (a.c.n_kv * a.s.group) + head) * D;
}
template <int D>
DF2_DEV float2* joint_stat(const PagedAttnArgs& a, int token, int head) {
  const long long heads = a.c.n_kv * a.s.group;
  return reinterpret_cast<float2*>(a.g.joint + a.rq.n_tokens * heads * D) + token * heads + head;
}
// Two parts of a row's softmax joined: factors of their outputs, so that those need no division, and the maximum and
// sum of both.
struct JointParts {
  float mine, other, m, l;
  DF2_DEV JointParts(float m0, float l0, float2 st) {
    m = fmaxf(m0, st.x);
    const float ref = m == -INFINITY ? 0.f : m;
    mine = ex2(m0 - ref), other = ex2(st.x - ref);
    l = l0 * mine + st.y * other;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (a NaN sum stays NaN)
    mine *= inv, other *= inv;
  }
  DF2_DEV float lse() const { return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945f; }
};

}  // namespace df2
