// The pages of a pool: argument blocks and launch interfaces.
#pragma once

#include "paged.h"

namespace df2 {

struct PagePool {
  int32_t* ref;    // [n_pages] holders
  int32_t* table;  // [n_rows][table_stride]
  long long table_stride;
  int n_pages, n_rows, max_pages, page_size;
};

struct PagesResizeArgs {
  PagePool p;
  int32_t* kv_len;
  const int32_t* new_len;
  int32_t* copies;  // [3][n_rows]
  int32_t* status;
};
cudaError_t launch_pages_resize(const PagesResizeArgs& a, cudaStream_t st);

struct PagesForkArgs {
  PagePool p;
  int n;
  const int32_t* parent;
  const int32_t* child;
  int32_t* kv_len;
  int32_t* status;
};
cudaError_t launch_pages_fork(const PagesForkArgs& a, cudaStream_t st);

constexpr int kLayersPerLaunch = 24;  // of a launch's arguments
struct LayerPools {
  PagedCache c[kLayersPerLaunch];
};
struct PagesCopyArgs {
  int n, head_dim, size;  // copies; bytes of an element
  const int32_t* copies;  // [3][n]
  int32_t* status;
};
cudaError_t launch_pages_copy(const PagesCopyArgs& a, const LayerPools& pools, int layers, cudaStream_t st);

struct PagedKeepArgs {
  PagedReq rq;
  int head_dim, size;
  const int32_t* keep;
  long long keep_stride;
  int max_keep;
  const int32_t* n_keep;
  int32_t* kv_out;  // null: not written
};
constexpr int kKeepMax = 64;
cudaError_t launch_paged_keep(const PagedKeepArgs& a, const LayerPools& pools, int layers, cudaStream_t st);

}  // namespace df2
