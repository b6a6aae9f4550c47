// Host-side checks that the calls on the paged cache share, and the handle.
#pragma once

#include <math.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>

#include "../../include/dflash2.h"
#include "paged.h"

struct dflash2_paged_handle {
  dflash2_paged_config cfg;
  int num_sms;
  float* part;
  int* desc;
  unsigned* count;
};

namespace df2 {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int kv_size(int fmt) { return fmt == DFLASH2_KV_BF16 || fmt == DFLASH2_KV_F16 ? 2 : 1; }
inline int t_size(int type) { return type == DFLASH2_T_F32 ? 4 : 2; }
inline bool quantised(int fmt) { return kv_size(fmt) == 1; }
// a stride in bytes: a whole number of 16-byte pieces (either sign)
inline bool stride16(int64_t elements, int size) { return (elements * size) % 16 == 0; }

inline bool valid_rows(const dflash2_rows& r) {
  return r.p && aligned16(r.p) && r.type >= DFLASH2_T_BF16 && r.type <= DFLASH2_T_F32 &&
         stride16(r.token_stride, t_size(r.type)) && stride16(r.head_stride, t_size(r.type));
}

// Whether no two of the rows share a channel: the step between two of them (dt tokens, dh heads) never comes to less than a row.
inline bool rows_apart(const dflash2_rows& r, int64_t tokens, int64_t heads, int64_t dim) {
  const int64_t t = std::abs(r.token_stride), h = std::abs(r.head_stride);
  if ((heads == 1 || h >= dim) && (tokens == 1 || t >= (heads - 1) * h + dim)) return true;   // heads within tokens
  if ((tokens == 1 || t >= dim) && (heads == 1 || h >= (tokens - 1) * t + dim)) return true;  // tokens within heads
  for (int64_t dh = 0; dh < heads; ++dh) {  // any other order: the tokens that come nearest to dh heads
    const int64_t near = t > 0 ? std::min(dh * h / t, tokens - 1) : 0;
    for (int64_t dt = near; dt <= near + 1; ++dt)
      if (dt < tokens && dt + dh > 0 && std::abs(dt * t - dh * h) < dim) return false;
  }
  return true;
}

inline PagedRows rows_of(const dflash2_rows& r) {
  return PagedRows{static_cast<char*>(r.p), r.token_stride, r.head_stride, r.type};
}

inline dflash2_status check_cache(const dflash2_paged_handle* h, const dflash2_paged_cache* c, int32_t n_req) {
  if (!h || !c || n_req < 0) return DFLASH2_E_INVAL;
  if (n_req > h->cfg.max_requests) return DFLASH2_E_UNSUPPORTED;
  if (n_req == 0) return DFLASH2_OK;  // (an empty batch's table has no address)
  const int size = kv_size(h->cfg.kv_format);
  if (!c->k || !c->v || !c->page_table || !aligned16(c->k) || !aligned16(c->v) || c->n_pages < 1 || c->max_pages < 1 ||
      c->table_stride < c->max_pages || !stride16(c->page_stride, size) || !stride16(c->token_stride, size) ||
      !stride16(c->head_stride, size))
    return DFLASH2_E_INVAL;
  if (quantised(h->cfg.kv_format) && (!c->k_scale || !c->v_scale)) return DFLASH2_E_INVAL;
  return DFLASH2_OK;
}

inline PagedCache cache_of(const dflash2_paged_handle* h, const dflash2_paged_cache* c) {
  PagedCache r;
  r.k = static_cast<char*>(c->k);
  r.v = static_cast<char*>(c->v);
  r.k_scale = c->k_scale;
  r.v_scale = c->v_scale;
  r.table = c->page_table;
  r.page_stride = c->page_stride;
  r.token_stride = c->token_stride;
  r.head_stride = c->head_stride;
  r.s_page_stride = c->scale_page_stride;
  r.s_token_stride = c->scale_token_stride;
  r.s_head_stride = c->scale_head_stride;
  r.table_stride = c->table_stride;
  r.n_pages = c->n_pages;
  r.max_pages = c->max_pages;
  r.page_size = h->cfg.page_size;
  r.n_kv = h->cfg.n_kv_heads;
  return r;
}

inline int capacity_of(const dflash2_paged_handle* h, const dflash2_paged_cache* c) {
  const int64_t cap = static_cast<int64_t>(c->max_pages) * h->cfg.page_size;
  return static_cast<int>(std::min<int64_t>(cap, kPagedMaxLen));
}

// The checks of an attention's arguments, and its kernels' arguments.  empty: there is nothing to do.
inline dflash2_status attention_args(const dflash2_paged_handle* h, const dflash2_paged_cache* cache,
                                     const dflash2_paged_attention_args& x, PagedAttnArgs* out, bool* empty) {
  const dflash2_status s = check_cache(h, cache, x.n_req);
  if (s != DFLASH2_OK) return s;
  if (x.n_tokens < 0 || x.max_new < 0 || x.max_len < 0 || (x.n_req > 0 && (!x.token_begin || !x.kv_len)) || x.window < 0 ||
      !isfinite(x.scale))
    return DFLASH2_E_INVAL;
  if (x.tree_mask && x.max_new > DFLASH2_PAGED_MAX_TREE) return DFLASH2_E_UNSUPPORTED;
  *empty = x.n_tokens == 0 || x.max_new == 0 || x.n_req == 0;
  if (*empty) return DFLASH2_OK;
  if (!valid_rows(x.q) || !valid_rows(x.out) || x.q.type != x.out.type || x.q.type == DFLASH2_T_F32)
    return DFLASH2_E_INVAL;
  if (!quantised(h->cfg.kv_format) && x.q.type != (h->cfg.kv_format == DFLASH2_KV_BF16 ? DFLASH2_T_BF16 : DFLASH2_T_F16))
    return DFLASH2_E_INVAL;
  if (static_cast<int64_t>(std::min(x.max_new, x.n_tokens)) * (h->cfg.n_q_heads / h->cfg.n_kv_heads) > kPagedMaxRows)
    return DFLASH2_E_UNSUPPORTED;
  PagedAttnArgs& a = *out;
  memset(&a, 0, sizeof(a));
  a.c = cache_of(h, cache);
  // no request can hold more than the call's rows, or more positions than its page table's row
  const int cap = capacity_of(h, cache);
  a.rq = PagedReq{x.token_begin, x.kv_len, x.status, x.n_req, x.n_tokens, std::min(x.max_new, x.n_tokens),
                  std::min(x.max_len, cap)};
  a.s.group = h->cfg.n_q_heads / h->cfg.n_kv_heads;
  a.s.causal = x.tree_mask ? 2 : (x.causal ? 1 : 0);
  a.s.window = std::min(x.window, 1 << 30);  // (differences of positions stay within 32 bits)
  a.q = rows_of(x.q);
  a.out = rows_of(x.out);
  a.tree = reinterpret_cast<const unsigned long long*>(x.tree_mask);
  a.lse = x.lse;
  a.scale_log2 = x.scale * 1.44269504f;
  a.part = h->part;
  a.desc = h->desc;
  a.count = h->count;
  return DFLASH2_OK;
}

}  // namespace df2
