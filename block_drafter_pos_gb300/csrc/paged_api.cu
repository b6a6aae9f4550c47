// Host side of the paged cache, its attention and the sampling: argument checks and launches.
// Nothing is allocated after dflash2_paged_create, and no call synchronises.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "../../include/dflash2.h"
#include "paged.h"
#include "sample.h"

using namespace df2;

static_assert(int(DFLASH2_KV_BF16) == int(kKvBf16) && int(DFLASH2_KV_F16) == int(kKvF16) &&
                  int(DFLASH2_KV_INT8) == int(kKvInt8) && int(DFLASH2_KV_E4M3) == int(kKvE4m3) &&
                  int(DFLASH2_T_BF16) == int(kTBf16) && int(DFLASH2_T_F16) == int(kTF16) && int(DFLASH2_T_F32) == int(kTF32),
              "the header's enumerations");

struct dflash2_paged_handle {
  dflash2_paged_config cfg;
  int num_sms;
  float* part;
  int* desc;
  unsigned* count;
};

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int kv_size(int fmt) { return fmt == DFLASH2_KV_BF16 || fmt == DFLASH2_KV_F16 ? 2 : 1; }
int t_size(int type) { return type == DFLASH2_T_F32 ? 4 : 2; }
bool quantised(int fmt) { return kv_size(fmt) == 1; }
// a stride in bytes: a whole number of 16-byte pieces (either sign)
bool stride16(int64_t elements, int size) { return (elements * size) % 16 == 0; }

bool valid_rows(const dflash2_rows& r) {
  return r.p && aligned16(r.p) && r.type >= DFLASH2_T_BF16 && r.type <= DFLASH2_T_F32 &&
         stride16(r.token_stride, t_size(r.type)) && stride16(r.head_stride, t_size(r.type));
}

PagedRows rows_of(const dflash2_rows& r) {
  return PagedRows{static_cast<char*>(r.p), r.token_stride, r.head_stride, r.type};
}

dflash2_status check_cache(const dflash2_paged_handle* h, const dflash2_paged_cache* c, int32_t n_req) {
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

PagedCache cache_of(const dflash2_paged_handle* h, const dflash2_paged_cache* c) {
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

int capacity_of(const dflash2_paged_handle* h, const dflash2_paged_cache* c) {
  const int64_t cap = static_cast<int64_t>(c->max_pages) * h->cfg.page_size;
  return static_cast<int>(std::min<int64_t>(cap, kPagedMaxLen));
}

dflash2_status move_rows(dflash2_paged_handle* h, const dflash2_paged_cache* cache, int32_t n_req, int32_t n_tokens,
                         const int32_t* token_begin, const int32_t* kv_len, const dflash2_rows* k,
                         const dflash2_rows* v, int32_t* status, void* stream, bool write) {
  const dflash2_status s = check_cache(h, cache, n_req);
  if (s != DFLASH2_OK) return s;
  if (n_tokens < 0 || !k || !v || (n_req > 0 && (!token_begin || !kv_len))) return DFLASH2_E_INVAL;
  if (n_tokens == 0 || n_req == 0) return DFLASH2_OK;
  if (!valid_rows(*k) || !valid_rows(*v) || k->type != v->type) return DFLASH2_E_INVAL;
  PagedMoveArgs a;
  a.c = cache_of(h, cache);
  a.rq = PagedReq{token_begin, kv_len, status, n_req, n_tokens, n_tokens, capacity_of(h, cache)};
  a.k = rows_of(*k);
  a.v = rows_of(*v);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = write ? launch_paged_write(a, h->cfg.head_dim, h->cfg.kv_format, st)
                              : launch_paged_read(a, h->cfg.head_dim, h->cfg.kv_format, st);
  return e == cudaSuccess ? DFLASH2_OK : DFLASH2_E_CUDA;
}

}  // namespace

extern "C" {

dflash2_status dflash2_paged_create(const dflash2_paged_config* cfg, dflash2_paged_handle** out) {
  if (!cfg || !out) return DFLASH2_E_INVAL;
  *out = nullptr;
  const dflash2_paged_config& c = *cfg;
  if (c.n_q_heads < 1 || c.n_kv_heads < 1 || c.head_dim < 1 || c.page_size < 1 || c.max_requests < 1 ||
      c.kv_format < DFLASH2_KV_BF16 || c.kv_format > DFLASH2_KV_E4M3)
    return DFLASH2_E_INVAL;
  if ((c.head_dim != 64 && c.head_dim != 128) || c.n_q_heads % c.n_kv_heads || c.n_q_heads / c.n_kv_heads > 64 ||
      c.n_kv_heads > 1024 || c.max_requests > DFLASH2_PAGED_MAX_REQUESTS)
    return DFLASH2_E_UNSUPPORTED;
  dflash2_paged_handle* h = new (std::nothrow) dflash2_paged_handle;
  if (!h) return DFLASH2_E_CUDA;
  memset(h, 0, sizeof(*h));
  h->cfg = c;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    delete h;
    return DFLASH2_E_CUDA;
  }
  // two partial slots per CTA of the attention, and the cut units' descriptions
  const size_t ctas = static_cast<size_t>(h->num_sms) * kPagedMaxCtasPerSm;
  static_assert(kChunkRows >= 64 * kPagedMaxCtasPerSm, "the larger scratch serves both kernels");
  const size_t part = paged_part_floats(h->num_sms, c.head_dim) * 4;
  char* p = nullptr;
  if (cudaMalloc(&p, part + ctas * 36) != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return DFLASH2_E_CUDA;
  }
  // (finished before the handle is used on any stream)
  if (cudaMemset(p + part, 0, ctas * 36) != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess) {
    cudaFree(p);
    delete h;
    return DFLASH2_E_CUDA;
  }
  h->part = reinterpret_cast<float*>(p);
  h->desc = reinterpret_cast<int*>(p + part);
  h->count = reinterpret_cast<unsigned*>(p + part + ctas * 32);
  *out = h;
  return DFLASH2_OK;
}

dflash2_status dflash2_paged_destroy(dflash2_paged_handle* h) {
  if (!h) return DFLASH2_E_INVAL;
  const cudaError_t e = cudaFree(h->part);
  delete h;
  return e == cudaSuccess ? DFLASH2_OK : DFLASH2_E_CUDA;
}

dflash2_status dflash2_paged_write(dflash2_paged_handle* h, const dflash2_paged_cache* cache, int32_t n_req,
                                   int32_t n_tokens, const int32_t* token_begin, const int32_t* kv_len,
                                   const dflash2_rows* k, const dflash2_rows* v, int32_t* status, void* stream) {
  return move_rows(h, cache, n_req, n_tokens, token_begin, kv_len, k, v, status, stream, true);
}

dflash2_status dflash2_paged_read(dflash2_paged_handle* h, const dflash2_paged_cache* cache, int32_t n_req,
                                  int32_t n_tokens, const int32_t* token_begin, const int32_t* kv_len,
                                  const dflash2_rows* k, const dflash2_rows* v, int32_t* status, void* stream) {
  return move_rows(h, cache, n_req, n_tokens, token_begin, kv_len, k, v, status, stream, false);
}

dflash2_status dflash2_paged_attention(dflash2_paged_handle* h, const dflash2_paged_cache* cache,
                                       const dflash2_paged_attention_args* args, void* stream) {
  if (!args) return DFLASH2_E_INVAL;
  const dflash2_paged_attention_args& x = *args;
  const dflash2_status s = check_cache(h, cache, x.n_req);
  if (s != DFLASH2_OK) return s;
  if (x.n_tokens < 0 || x.max_new < 0 || x.max_len < 0 || (x.n_req > 0 && (!x.token_begin || !x.kv_len)) || x.window < 0 ||
      !isfinite(x.scale))
    return DFLASH2_E_INVAL;
  if (x.tree_mask && x.max_new > DFLASH2_PAGED_MAX_TREE) return DFLASH2_E_UNSUPPORTED;
  if (x.n_tokens == 0 || x.max_new == 0 || x.n_req == 0) return DFLASH2_OK;
  if (!valid_rows(x.q) || !valid_rows(x.out) || x.q.type != x.out.type || x.q.type == DFLASH2_T_F32)
    return DFLASH2_E_INVAL;
  if (!quantised(h->cfg.kv_format) && x.q.type != (h->cfg.kv_format == DFLASH2_KV_BF16 ? DFLASH2_T_BF16 : DFLASH2_T_F16))
    return DFLASH2_E_INVAL;
  if (static_cast<int64_t>(std::min(x.max_new, x.n_tokens)) * (h->cfg.n_q_heads / h->cfg.n_kv_heads) > kPagedMaxRows)
    return DFLASH2_E_UNSUPPORTED;
  PagedAttnArgs a;
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
  const cudaError_t e = launch_paged_attention(a, h->cfg.head_dim, h->cfg.kv_format, x.q.type, h->num_sms,
                                               static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DFLASH2_OK : DFLASH2_E_CUDA;
}

dflash2_status dflash2_sample(const dflash2_sample_args* args, void* stream) {
  if (!args) return DFLASH2_E_INVAL;
  const dflash2_sample_args& x = *args;
  if (x.n_rows < 0 || x.vocab < 1 || x.logits_type < DFLASH2_T_BF16 || x.logits_type > DFLASH2_T_F32)
    return DFLASH2_E_INVAL;
  if (x.vocab > kSampleMaxVocab || x.n_rows > (1 << 24)) return DFLASH2_E_UNSUPPORTED;
  if (x.n_rows == 0) return DFLASH2_OK;
  if (!x.logits || !x.temperature || !x.uniform || !x.token || (x.n_rows > 1 && x.row_stride < x.vocab) ||
      (x.kept && x.n_rows > 1 && x.kept_stride < x.vocab) || reinterpret_cast<uintptr_t>(x.logits) % t_size(x.logits_type))
    return DFLASH2_E_INVAL;
  SampleArgs a;
  a.logits = x.logits;
  a.row_stride = x.row_stride;
  a.n_rows = x.n_rows;
  a.vocab = x.vocab;
  a.type = x.logits_type;
  a.temperature = x.temperature;
  a.top_k = x.top_k;
  a.top_p = x.top_p;
  a.min_p = x.min_p;
  a.uniform = x.uniform;
  a.token = x.token;
  a.prob = x.prob;
  a.kept = x.kept;
  a.kept_stride = x.kept_stride;
  a.status = x.status;
  const char *l0 = static_cast<const char*>(x.logits), *k0 = reinterpret_cast<const char*>(x.kept);
  const int64_t lb = ((x.n_rows - 1) * x.row_stride + x.vocab) * t_size(x.logits_type);
  const int64_t kb = ((x.n_rows - 1) * x.kept_stride + x.vocab) * 4;
  a.kept_in_place = k0 != nullptr && k0 < l0 + lb && l0 < k0 + kb;
  // in place: the same rows, or one row's kept logits would overwrite another's before they are read
  if (a.kept_in_place && (k0 != l0 || x.logits_type != DFLASH2_T_F32 || (x.n_rows > 1 && x.kept_stride != x.row_stride)))
    return DFLASH2_E_INVAL;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&a.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return DFLASH2_E_CUDA;
  return launch_sample(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DFLASH2_OK : DFLASH2_E_CUDA;
}

}  // extern "C"
