// Host side of rotary positions, the pages of a pool, and attention over shared prefixes: argument checks and launches.
// Nothing is allocated, and no call synchronises.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "../../include/dflash2.h"
#include "pages.h"
#include "paged_api.h"
#include "rope.h"

using namespace df2;

static_assert(DFLASH2_ROPE_MAX_DIM == 2 * kRopeMaxPairs && DFLASH2_PAGED_MAX_TREE == kKeepMax &&
                  int(DFLASH2_SHARED_AUTO) == int(kSharedAuto) && int(DFLASH2_SHARED_TOGETHER) == int(kSharedTogether) &&
                  int(DFLASH2_SHARED_APART) == int(kSharedApart),
              "the header's limits and enumerations");

namespace {

bool sm_count(int* n) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

// Whether a plan is one that dflash2_rope_plan may have made.
bool valid_plan(const dflash2_rotation* r) {
  return r && r->rot_dim >= 16 && r->rot_dim <= DFLASH2_ROPE_MAX_DIM && r->rot_dim % 16 == 0 &&
         (r->interleaved == 0 || r->interleaved == 1) && isfinite(r->amplitude);
}

RopePlan plan_of(const dflash2_rotation& r, bool inverse) {
  RopePlan p;
  p.rot = r.rot_dim;
  p.interleaved = r.interleaved;
  p.amplitude = r.amplitude;
  p.sign = inverse ? -1.f : 1.f;
  static_assert(sizeof(p.turns) == sizeof(r.turns), "pairs");
  memcpy(p.turns, r.turns, sizeof(p.turns));
  return p;
}

// The bytes that rows reach over, [lo, hi).
void span_of(const dflash2_rows& r, int64_t tokens, int64_t heads, int64_t dim, const char** lo, const char** hi) {
  const int64_t t = (tokens - 1) * r.token_stride, h = (heads - 1) * r.head_stride, size = t_size(r.type);
  *lo = static_cast<const char*>(r.p) + (std::min<int64_t>(t, 0) + std::min<int64_t>(h, 0)) * size;
  *hi = static_cast<const char*>(r.p) + (std::max<int64_t>(t, 0) + std::max<int64_t>(h, 0) + dim) * size;
}

// Rows that may be turned from x to y: of one type, and apart from each other or the same; no two of y's overlap.
bool valid_turn(const dflash2_rows* x, const dflash2_rows* y, int64_t tokens, int64_t heads, int64_t dim) {
  if (!x || !y || !valid_rows(*x) || !valid_rows(*y) || x->type != y->type || !rows_apart(*y, tokens, heads, dim)) return false;
  if (x->p == y->p && x->token_stride == y->token_stride && x->head_stride == y->head_stride) return true;
  const char *x0, *x1, *y0, *y1;
  span_of(*x, tokens, heads, dim, &x0, &x1);
  span_of(*y, tokens, heads, dim, &y0, &y1);
  return x1 <= y0 || y1 <= x0;
}

// Layers' pools, 24 at a launch.
template <typename F>
dflash2_status by_layers(const dflash2_paged_handle* h, int32_t n_caches, const dflash2_paged_cache* caches, F launch) {
  for (int l = 0; l < n_caches; l += kLayersPerLaunch) {
    LayerPools pools;
    const int n = std::min(kLayersPerLaunch, n_caches - l);
    for (int i = 0; i < n; ++i) pools.c[i] = cache_of(h, caches + l + i);
    if (launch(pools, n) != cudaSuccess) return DFLASH2_E_CUDA;
  }
  return DFLASH2_OK;
}

dflash2_status check_pool(const dflash2_page_pool* p) {
  if (!p || p->n_pages < 1 || p->n_rows < 0 || p->max_pages < 1 || p->page_size < 1 || p->table_stride < p->max_pages)
    return DFLASH2_E_INVAL;
  if (p->n_pages > DFLASH2_PAGES_MAX || p->n_rows > DFLASH2_PAGED_MAX_REQUESTS) return DFLASH2_E_UNSUPPORTED;
  if (p->n_rows == 0) return DFLASH2_OK;  // (an empty table has no address)
  return p->ref && p->page_table ? DFLASH2_OK : DFLASH2_E_INVAL;
}

PagePool pool_of(const dflash2_page_pool& p) {
  return PagePool{p.ref, p.page_table, p.table_stride, p.n_pages, p.n_rows, p.max_pages, p.page_size};
}

}  // namespace

extern "C" {

dflash2_status dflash2_rope_plan(const dflash2_rope_config* cfg, dflash2_rotation* out) {
  if (!cfg || !out) return DFLASH2_E_INVAL;
  const dflash2_rope_config& c = *cfg;
  memset(out, 0, sizeof(*out));
  const bool yarn = c.scaling == DFLASH2_ROPE_YARN;
  if (c.rot_dim < 1 || (c.interleaved != 0 && c.interleaved != 1) || c.scaling < DFLASH2_ROPE_PLAIN ||
      c.scaling > DFLASH2_ROPE_TABLE || !isfinite(c.amplitude) || c.amplitude < 0)
    return DFLASH2_E_INVAL;
  if (c.scaling == DFLASH2_ROPE_TABLE ? !c.table : !isfinite(c.theta) || c.theta <= 1) return DFLASH2_E_INVAL;
  if ((c.scaling == DFLASH2_ROPE_LINEAR && (!isfinite(c.factor) || c.factor <= 0)) ||
      (yarn && (!isfinite(c.factor) || c.factor < 1 || c.original_len < 1 || !isfinite(c.beta_fast) || c.beta_fast < 0 ||
                !isfinite(c.beta_slow) || c.beta_slow < 0)))
    return DFLASH2_E_INVAL;
  if (c.rot_dim % 16 || c.rot_dim > DFLASH2_ROPE_MAX_DIM) return DFLASH2_E_UNSUPPORTED;
  const double pi = 3.14159265358979323846, rot = c.rot_dim;
  double lo = 0, hi = 0;
  if (yarn) {
    auto pair_of = [&](double turns) { return rot * log(c.original_len / (turns * 2 * pi)) / (2 * log(c.theta)); };
    lo = std::max(floor(pair_of(c.beta_fast > 0 ? c.beta_fast : 32)), 0.0);
    hi = std::min(ceil(pair_of(c.beta_slow > 0 ? c.beta_slow : 1)), rot - 1);
  }
  double rate[DFLASH2_ROPE_MAX_DIM / 2];
  for (int i = 0; i < c.rot_dim / 2; ++i) {
    double f = c.scaling == DFLASH2_ROPE_TABLE ? c.table[i] : pow(c.theta, -2.0 * i / rot);
    if (c.scaling == DFLASH2_ROPE_LINEAR) f /= c.factor;
    if (yarn) {
      const double g = std::min(std::max((i - lo) / (hi > lo ? hi - lo : 0.001), 0.0), 1.0);
      f = f * (1 - g) + f / c.factor * g;
    }
    if (!(fabs(f) <= 1048576.0)) return DFLASH2_E_INVAL;
    rate[i] = f;
  }
  const float amplitude = static_cast<float>(c.amplitude > 0 ? c.amplitude : (yarn ? 0.1 * log(c.factor) + 1 : 1.0));
  if (!isfinite(amplitude)) return DFLASH2_E_INVAL;
  out->rot_dim = c.rot_dim;
  out->interleaved = c.interleaved;
  out->amplitude = amplitude;
  for (int i = 0; i < c.rot_dim / 2; ++i) {
    const double t = rate[i] / (2 * pi), f = t - floor(t);  // [0, 1] (1 for a tiny negative rate: no turn)
    const double high = floor(f * 4294967296.0);
    const double low = (f * 4294967296.0 - high) * 4294967296.0;
    out->turns[i] = (static_cast<uint64_t>(high) << 32) + static_cast<uint64_t>(low);
  }
  return DFLASH2_OK;
}

dflash2_status dflash2_rope(const dflash2_rotation* rope, int32_t n_tokens, int32_t head_dim, int32_t x_heads,
                            const dflash2_rows* x, const dflash2_rows* out, int32_t k_heads, const dflash2_rows* k,
                            const dflash2_rows* k_out, const int32_t* positions, int32_t inverse, void* stream) {
  if (!valid_plan(rope) || n_tokens < 0 || x_heads < 0 || k_heads < 0 || head_dim < 8) return DFLASH2_E_INVAL;
  if (head_dim % 8 || head_dim > kRopeMaxDim || head_dim < rope->rot_dim || x_heads > kRopeMaxHeads || k_heads > kRopeMaxHeads - x_heads ||
      n_tokens > kRopeMaxTokens)
    return DFLASH2_E_UNSUPPORTED;
  if (n_tokens == 0 || x_heads + k_heads == 0) return DFLASH2_OK;
  if (!positions || (x_heads > 0 && !valid_turn(x, out, n_tokens, x_heads, head_dim)) ||
      (k_heads > 0 && !valid_turn(k, k_out, n_tokens, k_heads, head_dim)) || (x_heads > 0 && k_heads > 0 && x->type != k->type))
    return DFLASH2_E_INVAL;
  RopeArgs a;
  memset(&a, 0, sizeof(a));
  if (x_heads > 0) a.x = rows_of(*x), a.y = rows_of(*out);
  if (k_heads > 0) a.k = rows_of(*k), a.ky = rows_of(*k_out);
  if (x_heads == 0) a.x.type = a.k.type;
  a.n_tokens = n_tokens;
  a.dim = head_dim;
  a.x_heads = x_heads;
  a.k_heads = k_heads;
  a.x_copy = a.x.p != a.y.p;
  a.k_copy = a.k.p != a.ky.p;
  a.positions = positions;
  a.plan = plan_of(*rope, inverse != 0);
  int num_sms = 0;
  if (!sm_count(&num_sms)) return DFLASH2_E_CUDA;
  return launch_rope(a, num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DFLASH2_OK : DFLASH2_E_CUDA;
}

dflash2_status dflash2_paged_rope_write(dflash2_paged_handle* h, const dflash2_rotation* rope,
                                        const dflash2_paged_cache* cache, int32_t n_req, int32_t n_tokens,
                                        const int32_t* token_begin, const int32_t* kv_len, const int32_t* positions,
                                        const dflash2_rows* q, const dflash2_rows* q_out, const dflash2_rows* k,
                                        const dflash2_rows* v, int32_t* status, void* stream) {
  const dflash2_status s = check_cache(h, cache, n_req);
  if (s != DFLASH2_OK) return s;
  if (!valid_plan(rope) || n_tokens < 0 || !k || !v || (n_req > 0 && (!token_begin || !kv_len))) return DFLASH2_E_INVAL;
  if (rope->rot_dim > h->cfg.head_dim || n_tokens > kRopeMaxTokens) return DFLASH2_E_UNSUPPORTED;
  if (n_tokens == 0 || n_req == 0) return DFLASH2_OK;
  if (!valid_rows(*k) || !valid_rows(*v) || k->type != v->type) return DFLASH2_E_INVAL;
  if (q && (!valid_turn(q, q_out, n_tokens, h->cfg.n_q_heads, h->cfg.head_dim) || q->type != k->type)) return DFLASH2_E_INVAL;
  RopeWriteArgs a;
  memset(&a, 0, sizeof(a));
  a.move.c = cache_of(h, cache);
  a.move.rq = PagedReq{token_begin, kv_len, status, n_req, n_tokens, n_tokens, capacity_of(h, cache)};
  a.move.k = rows_of(*k);
  a.move.v = rows_of(*v);
  if (q) {
    a.q = rows_of(*q);
    a.y = rows_of(*q_out);
    a.q_heads = h->cfg.n_q_heads;
    a.q_copy = a.q.p != a.y.p;
  }
  a.positions = positions;
  a.plan = plan_of(*rope, false);
  const cudaError_t e = launch_rope_write(a, h->cfg.head_dim, h->cfg.kv_format, h->num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DFLASH2_OK : DFLASH2_E_CUDA;
}

dflash2_status dflash2_pages_resize(const dflash2_page_pool* pool, int32_t* kv_len, const int32_t* new_len,
                                    int32_t* copies, int32_t* status, void* stream) {
  const dflash2_status s = check_pool(pool);
  if (s != DFLASH2_OK || pool->n_rows == 0) return s;
  if (!kv_len || !new_len || !copies || kv_len == new_len) return DFLASH2_E_INVAL;
  const PagesResizeArgs a{pool_of(*pool), kv_len, new_len, copies, status};
  return launch_pages_resize(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DFLASH2_OK : DFLASH2_E_CUDA;
}

dflash2_status dflash2_pages_fork(const dflash2_page_pool* pool, int32_t n_fork, const int32_t* parent,
                                  const int32_t* child, int32_t* kv_len, int32_t* status, void* stream) {
  const dflash2_status s = check_pool(pool);
  if (s != DFLASH2_OK) return s;
  if (n_fork < 0) return DFLASH2_E_INVAL;
  if (n_fork > DFLASH2_PAGED_MAX_REQUESTS) return DFLASH2_E_UNSUPPORTED;
  if (n_fork == 0) return DFLASH2_OK;
  if (!parent || !child || pool->n_rows == 0 || !kv_len) return DFLASH2_E_INVAL;
  const PagesForkArgs a{pool_of(*pool), n_fork, parent, child, kv_len, status};
  return launch_pages_fork(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DFLASH2_OK : DFLASH2_E_CUDA;
}

dflash2_status dflash2_pages_copy(dflash2_paged_handle* h, int32_t n_caches, const dflash2_paged_cache* caches,
                                  int32_t n, const int32_t* copies, int32_t* status, void* stream) {
  if (!h || n_caches < 0 || n < 0 || (n_caches > 0 && !caches)) return DFLASH2_E_INVAL;
  if (n > (1 << 20)) return DFLASH2_E_UNSUPPORTED;
  for (int l = 0; l < n_caches; ++l) {
    dflash2_paged_cache c = caches[l];
    if (!c.page_table) c.page_table = reinterpret_cast<const int32_t*>(16);  // (not looked at)
    c.max_pages = std::max(c.max_pages, 1);
    c.table_stride = std::max<int64_t>(c.table_stride, c.max_pages);
    const dflash2_status s = check_cache(h, &c, 1);
    if (s != DFLASH2_OK) return s;
  }
  if (n == 0 || n_caches == 0) return DFLASH2_OK;
  if (!copies) return DFLASH2_E_INVAL;
  const PagesCopyArgs a{n, h->cfg.head_dim, kv_size(h->cfg.kv_format), copies, status};
  return by_layers(h, n_caches, caches,
                   [&](const LayerPools& p, int layers) { return launch_pages_copy(a, p, layers, static_cast<cudaStream_t>(stream)); });
}

dflash2_status dflash2_paged_keep(dflash2_paged_handle* h, int32_t n_caches, const dflash2_paged_cache* caches,
                                  int32_t n_req, const int32_t* token_begin, const int32_t* kv_len,
                                  const int32_t* keep, int64_t keep_stride, int32_t max_keep, const int32_t* n_keep,
                                  int32_t* kv_out, int32_t* status, void* stream) {
  if (!h || n_caches < 1 || !caches || max_keep < 0 || (n_req > 1 && keep_stride < max_keep)) return DFLASH2_E_INVAL;
  for (int l = 0; l < n_caches; ++l) {
    const dflash2_status s = check_cache(h, caches + l, n_req);
    if (s != DFLASH2_OK) return s;
  }
  if (n_req == 0) return DFLASH2_OK;
  if (!token_begin || !kv_len || (max_keep > 0 && !keep) || !n_keep || kv_out == kv_len) return DFLASH2_E_INVAL;
  PagedKeepArgs a;
  a.rq = PagedReq{token_begin, kv_len, status, n_req, 0x7FFFFFFF, kKeepMax, kPagedMaxLen};
  a.head_dim = h->cfg.head_dim;
  a.size = kv_size(h->cfg.kv_format);
  a.keep = keep;
  a.keep_stride = keep_stride;
  a.max_keep = max_keep;
  a.n_keep = n_keep;
  a.kv_out = kv_out;
  return by_layers(h, n_caches, caches,
                   [&](const LayerPools& p, int layers) { return launch_paged_keep(a, p, layers, static_cast<cudaStream_t>(stream)); });
}

int64_t dflash2_paged_shared_bytes(const dflash2_paged_handle* h, int32_t n_tokens) {
  if (!h || n_tokens < 0) return 0;
  return static_cast<int64_t>(n_tokens) * h->cfg.n_q_heads * (h->cfg.head_dim + 2) * 4;
}

dflash2_status dflash2_paged_attention_shared(dflash2_paged_handle* h, const dflash2_paged_cache* cache,
                                              const dflash2_paged_shared_args* args, void* stream) {
  if (!args) return DFLASH2_E_INVAL;
  const dflash2_paged_shared_args& x = *args;
  PagedAttnArgs a;
  bool empty = false;
  const dflash2_status s = attention_args(h, cache, x.x, &a, &empty);
  if (s != DFLASH2_OK) return s;
  if (x.n_groups < 0 || x.max_group < 0 || x.max_prefix < 0 || x.x.window != 0 || x.how < DFLASH2_SHARED_AUTO ||
      x.how > DFLASH2_SHARED_APART)
    return DFLASH2_E_INVAL;
  if (x.n_groups > DFLASH2_PAGED_MAX_REQUESTS) return DFLASH2_E_UNSUPPORTED;
  if (empty) return DFLASH2_OK;
  if (x.n_groups < 1 || !x.group_begin || !x.prefix_len) return DFLASH2_E_INVAL;
  const int max_group = std::min(x.max_group, x.x.n_tokens);
  if (static_cast<int64_t>(max_group) * a.s.group > kPagedMaxRows) return DFLASH2_E_UNSUPPORTED;
  if (!x.workspace || (reinterpret_cast<uintptr_t>(x.workspace) & 31u) != 0 || x.workspace_bytes < dflash2_paged_shared_bytes(h, x.x.n_tokens)) return DFLASH2_E_INVAL;
  a.g.begin = x.group_begin;
  a.g.prefix = x.prefix_len;
  a.g.n_groups = x.n_groups;
  a.g.n_req = x.x.n_req;
  a.g.max_group = max_group;
  a.g.max_prefix = std::min(x.max_prefix, capacity_of(h, cache));
  a.g.apart = x.how;
  a.g.joint = static_cast<float*>(x.workspace);
  const cudaError_t e = launch_shared_attention(a, h->cfg.head_dim, h->cfg.kv_format, x.x.q.type, h->num_sms,
                                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DFLASH2_OK : DFLASH2_E_CUDA;
}

}  // extern "C"
