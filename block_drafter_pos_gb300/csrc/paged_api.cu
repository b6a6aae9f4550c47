// Host side of the paged cache, its attention and the sampling: argument checks and launches.
// Nothing is allocated after dflash2_paged_create, and no call synchronises.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "../../include/dflash2.h"
#include "paged.h"
#include "paged_api.h"
#include "sample.h"

using namespace df2;

static_assert(int(DFLASH2_KV_BF16) == int(kKvBf16) && int(DFLASH2_KV_F16) == int(kKvF16) &&
                  int(DFLASH2_KV_INT8) == int(kKvInt8) && int(DFLASH2_KV_E4M3) == int(kKvE4m3) &&
                  int(DFLASH2_T_BF16) == int(kTBf16) && int(DFLASH2_T_F16) == int(kTF16) && int(DFLASH2_T_F32) == int(kTF32),
              "the header's enumerations");

namespace {

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
  PagedAttnArgs a;
  bool empty = false;
  const dflash2_status s = attention_args(h, cache, *args, &a, &empty);
  if (s != DFLASH2_OK || empty) return s;
  const cudaError_t e = launch_paged_attention(a, h->cfg.head_dim, h->cfg.kv_format, args->q.type, h->num_sms,
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
