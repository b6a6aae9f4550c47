// The pages of a pool that the rows of a page table share: taking and giving back, forking, copying, and moving a tree's
// accepted tokens together.
//
// State is the number of holders of each page, nothing else: a page without one is free, and the lowest free ids go
// first, so the result does not depend on the order of the device's work, and pages taken and given back leave the
// state as it was.  These are latencies, not bytes: each call is one launch.  Measured (us, profiled alone): eight rows
// of 63 pages grown and forked 9 and 4; 264 rows over 118,000 pages grown by 44 pages each 16, forked (256,000 holders) 7, freed 28;
// 255 tails of pages of one head copied 5.  Half of 256 rows of 44 pages grown while the other half is cut: 12.8, of which 0.9 is the
// barrier between giving back and taking.  255 tails of 32 positions of 8 heads of 128 in two layers: fp16 (134 MB) 28, 4.8 TB/s, 8-bit
// codes and scales 17.  Kept nodes of 48 trees in 16 layers (54 MB) 10 us, 5.3 TB/s.
#include <algorithm>

#include "common.cuh"
#include "pages.h"

namespace df2 {
namespace {

constexpr int kInval = 1, kNoPages = 5;  // DFLASH2_E_INVAL, DFLASH2_E_NO_PAGES

DF2_DEV int pages_of(int len, int page_size) { return len > 0 ? (len - 1) / page_size + 1 : 0; }
DF2_DEV bool in_pool(const PagePool& p, int page) { return page >= 0 && page < p.n_pages; }
DF2_DEV void flag(int32_t* status, int r, int what) {
  if (status) status[r] = what;
}
// One holder less; false if there was none.
DF2_DEV bool give_back(const PagePool& p, int page) {
  if (atomicSub(p.ref + page, 1) >= 1) return true;
  atomicAdd(p.ref + page, 1);
  return false;
}

// ------------------------------------------------------------------ taking and giving back
// A cluster of 16 CTAs (of 8: 256 samples freed, forked and grown 43 us against 41).  Every CTA works out what each row
// wants (a thread per row).  The counts are read in chunks of 1024 pages, a warp each, dealt to the CTAs in turn; each keeps its
// chunks' free pages as bits and tells all CTAs how many they are.  After the cluster's barrier nothing is read any more that
// the call changes: rows give back what they no longer hold, and each warp hands its chunks' free pages to the rows that
// their ranks fall to.
constexpr int kCluster = 16, kResizeThreads = 1024, kChunk = 1024;

DF2_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
DF2_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
DF2_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Writes to the same place of another CTA's shared memory.
DF2_DEV void put_remote(const int* place, uint32_t cta, int value) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.u32 [a], %2;\n}\n" ::"r"(
          static_cast<uint32_t>(__cvta_generic_to_shared(place))),
      "r"(cta), "r"(value)
      : "memory");
}

// Exclusive sum over the block of 1024 threads; `total` to all.  tmp: 33 words.
DF2_DEV long long block_scan(long long v, long long* tmp, long long& total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[wid] = x;
  __syncthreads();
  if (wid == 0) {
    const long long w = tmp[lane];
    long long s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    tmp[lane] = s - w;
    if (lane == 31) tmp[32] = s;
  }
  __syncthreads();
  const long long before = tmp[wid] + x - v;
  total = tmp[32];
  __syncthreads();
  return before;
}

constexpr int kSlots = 2 * kResizeThreads;  // (never more than half full)
static_assert(kSlots == 1 << 11, "the slot's bits of a product");
struct ResizeShared {
  long long tmp[33];
  int first[kResizeThreads + 1];  // rank of the first page a row takes (at most 2^30)
  int col[kResizeThreads];        // the column it goes to
  int tail[kResizeThreads];       // the last page, partly filled, of a row that grows; -1: none
  int what[kResizeThreads];       // bits below
  int served;                     // pages that rows take
  int key[kSlots], same[kSlots];  // rows with the tail `key`: how many,
  unsigned long long keeper[kSlots];  // and which of them has most positions there (the first of those): positions, 1023 - row
};
constexpr int kGood = 1, kRenews = 2, kServed = 4;

__global__ void __launch_bounds__(kResizeThreads, 1) resize_kernel(const __grid_constant__ PagesResizeArgs a) {
  extern __shared__ __align__(16) char smem[];
  ResizeShared& s = *reinterpret_cast<ResizeShared*>(smem);
  const PagePool& p = a.p;
  const int chunks = (p.n_pages + kChunk - 1) / kChunk;
  int* const count = reinterpret_cast<int*>(smem + sizeof(ResizeShared));        // [chunks], then the free pages before each
  uint32_t* const bits = reinterpret_cast<uint32_t*>(count + chunks);            // [own chunks][32]
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, cta = static_cast<int>(cluster_rank());

  cluster_arrive();  // (its shared memory may be written once a CTA has begun)
  // ---- what row tid wants
  int want = 0, what = 0, col = 0, tail = -1, holders = 0;
  bool cut = false;
  unsigned long long place = 0;
  if (tid < p.n_rows) {
    const int old = a.kv_len[tid], len = __ldg(a.new_len + tid);
    const int have = pages_of(old, p.page_size), need = pages_of(len, p.page_size);
    if (old >= 0 && len >= 0 && have <= p.max_pages && need <= p.max_pages) {
      what = kGood;
      cut = have > need;
      if (len > old) {
        want = need - have;
        col = have;
        if (old % p.page_size) {
          tail = p.table[tid * p.table_stride + have - 1];
          holders = in_pool(p, tail) ? p.ref[tail] : 0;
          if (holders < 1) tail = -1, want = 0, what = 0;
          place = static_cast<unsigned long long>(old % p.page_size) * kResizeThreads + (kResizeThreads - 1 - tid);
        }
      }
    }
  }
  s.tail[tid] = tail;
  for (int i = tid; i < kSlots; i += kResizeThreads) s.key[i] = -1, s.same[i] = 0, s.keeper[i] = 0;
  if (tid == 0) s.served = 0;
  __syncthreads();
  // Rows with one tail meet in a slot of a small table, where they are counted.  If all holders grow, the one that has most
  // positions in the page keeps it: what it writes lies behind all others' positions, whether or not those are served.
  int slot = -1;
  if (tail >= 0 && holders > 1) {
    slot = static_cast<int>((static_cast<uint32_t>(tail) * 2654435761u) >> 21);
    for (;; slot = (slot + 1) & (kSlots - 1)) {
      const int k = atomicCAS(&s.key[slot], -1, tail);
      if (k == -1 || k == tail) break;
    }
    atomicAdd(&s.same[slot], 1);
    atomicMax(&s.keeper[slot], place);
  }
  const bool cuts = __syncthreads_or(cut);  // (the same in every CTA)
  if (slot >= 0 && (s.keeper[slot] != place || s.same[slot] < holders)) what |= kRenews, ++want, --col;
  long long total;
  const long long before = block_scan(want, s.tmp, total);
  s.first[tid] = static_cast<int>(min(before, 1ll << 30));
  s.col[tid] = col;
  if (tid == 0) s.first[kResizeThreads] = static_cast<int>(min(total, 1ll << 30));

  // ---- the free pages
  cluster_wait();
  if (total > 0) {
    for (int k = cta + kCluster * wid; k < chunks; k += kCluster * (kResizeThreads / 32)) {
      uint32_t word = 0;
#pragma unroll
      for (int w0 = 0; w0 < 32; w0 += 16) {
        int v[16];
#pragma unroll
        for (int w = 0; w < 16; ++w) {
          const int page = k * kChunk + (w0 + w) * 32 + lane;
          v[w] = page < p.n_pages ? p.ref[page] : 1;
        }
#pragma unroll
        for (int w = 0; w < 16; ++w) {
          const uint32_t b = __ballot_sync(0xffffffffu, v[w] == 0);
          if (lane == w0 + w) word = b;
        }
      }
      bits[(k / kCluster) * 32 + lane] = word;
      const int n = __reduce_add_sync(0xffffffffu, __popc(word));
      if (lane < kCluster) put_remote(count + k, lane, n);
    }
  }
  cluster_arrive();
  cluster_wait();

  // ---- who is served: rows in order, as far as the free pages go
  if (total > 0) {
    const int each = (chunks + kResizeThreads - 1) / kResizeThreads;
    long long mine = 0, free_pages;
    for (int i = 0; i < each; ++i)
      if (tid * each + i < chunks) mine += count[tid * each + i];
    int at = static_cast<int>(block_scan(mine, s.tmp, free_pages));
    for (int i = 0; i < each; ++i)
      if (tid * each + i < chunks) {
        const int n = count[tid * each + i];
        count[tid * each + i] = at;
        at += n;
      }
    if (want == 0 || before + want <= free_pages) {
      what |= kServed;
      if (want > 0) atomicMax(&s.served, static_cast<int>(before + want));
    }
  } else {
    what |= kServed;
  }
  s.what[tid] = what;
  __syncthreads();

  // ---- what rows no longer hold, and their lengths (a warp per row)
  for (int r = cta + kCluster * wid; r < p.n_rows; r += kCluster * (kResizeThreads / 32)) {
    const int w = s.what[r], old = a.kv_len[r], len = __ldg(a.new_len + r);
    const bool done = (w & kGood) && (w & kServed);
    bool fine = true;
    if (done && len < old) {
      // (eight columns a lane in flight: what this costs is the latency of the loads and of the counts)
      const int end = pages_of(old, p.page_size);
      int32_t* const row = p.table + r * p.table_stride;
      for (int c = pages_of(len, p.page_size) + lane; c < end; c += 8 * 32) {
        int page[8], had[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) page[i] = c + 32 * i < end ? row[c + 32 * i] : -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) had[i] = in_pool(p, page[i]) ? atomicSub(p.ref + page[i], 1) : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (c + 32 * i >= end) continue;
          row[c + 32 * i] = -1;
          if (had[i] >= 1) continue;
          fine = false;
          if (in_pool(p, page[i])) atomicAdd(p.ref + page[i], 1);
        }
      }
    }
    fine = __all_sync(0xffffffffu, fine);
    if (lane == 0) {
      const bool copy = done && (w & kRenews);
      a.copies[r] = copy ? s.tail[r] : -1;
      if (!copy) a.copies[p.n_rows + r] = -1;
      a.copies[2 * p.n_rows + r] = copy ? old % p.page_size : 0;
      if (copy) fine = give_back(p, s.tail[r]);
      if (done) a.kv_len[r] = len;
      if (!(w & kGood) || !fine) flag(a.status, r, kInval);
      else if (!done) flag(a.status, r, kNoPages);
    }
  }

  // ---- pages to rows.  Not before all pages are given back: one that a row lists and does not hold may be among the free ones, and
  // its count would be taken for that row's.
  const int served = s.served;
  if (cuts && served > 0) {
    cluster_arrive();
    cluster_wait();
  }
  if (served > 0) {
    for (int k = cta + kCluster * wid; k < chunks; k += kCluster * (kResizeThreads / 32)) {
      int j = count[k];
      if (j >= served) break;
      uint32_t word = bits[(k / kCluster) * 32 + lane];
      int x = __popc(word);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      j += x - __popc(word);
      if (word == 0 || j >= served) continue;
      int r = 0, hi = kResizeThreads;  // the last row whose first page's rank is at most j (those that take none are passed over)
      while (hi - r > 1) {
        const int mid = (r + hi) >> 1;
        if (s.first[mid] <= j) r = mid;
        else hi = mid;
      }
      for (; word != 0 && j < served; word &= word - 1, ++j) {
        while (j >= s.first[r + 1]) ++r;
        const int page = k * kChunk + lane * 32 + __ffs(word) - 1, i = j - s.first[r];
        p.table[r * p.table_stride + s.col[r] + i] = page;
        p.ref[page] = 1;
        if (i == 0 && (s.what[r] & kRenews)) a.copies[p.n_rows + r] = page;
      }
    }
  }
}

// ------------------------------------------------------------------ forking: a CTA per pair
__global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ PagesForkArgs a) {
  const PagePool& p = a.p;
  const int i = blockIdx.x, from = __ldg(a.parent + i), to = __ldg(a.child + i);
  bool bad = from < 0 || from >= p.n_rows || to < 0 || to >= p.n_rows;
  // (each pair looks at all: none reads a length that another pair writes)
  for (int j = threadIdx.x; j < a.n && !bad; j += 256) {
    const int c = __ldg(a.child + j);
    bad = (j != i && c == to) || c == from || __ldg(a.parent + j) == to;
  }
  bad = __syncthreads_or(bad);
  int len = 0, have = 0;
  if (!bad) {
    len = a.kv_len[from];
    have = pages_of(len, p.page_size);
    bad = len < 0 || have > p.max_pages || a.kv_len[to] != 0;
    const int32_t* const row = p.table + from * p.table_stride;
    for (int c = threadIdx.x; c < have && !bad; c += 256) bad = !in_pool(p, row[c]);
    bad = __syncthreads_or(bad);
  }
  if (bad) {
    if (threadIdx.x == 0) flag(a.status, i, kInval);
    return;
  }
  const int32_t* const row = p.table + from * p.table_stride;
  int32_t* const out = p.table + to * p.table_stride;
  for (int c = threadIdx.x; c < have; c += 256) {
    const int page = row[c];
    out[c] = page;
    atomicAdd(p.ref + page, 1);
  }
  if (threadIdx.x == 0) a.kv_len[to] = len;
}

// ------------------------------------------------------------------ copying pages
// A CTA takes up to 1024 pieces of 16 bytes of one side of a page (four loads in flight a thread); blockIdx.y: the layer.
constexpr int kCopyPieces = 1024;

__global__ void __launch_bounds__(256) copy_kernel(const __grid_constant__ PagesCopyArgs a, const __grid_constant__ LayerPools l,
                                                   int parts) {
  const PagedCache& c = l.c[blockIdx.y];
  const int i = blockIdx.x / (2 * parts), side = (blockIdx.x / parts) & 1, part = blockIdx.x % parts;
  const int src = __ldg(a.copies + i), dst = __ldg(a.copies + a.n + i), rows = __ldg(a.copies + 2ll * a.n + i);
  if (src < 0 || dst < 0) return;
  if (src >= c.n_pages || dst >= c.n_pages || rows < 0 || rows > c.page_size) {
    if (threadIdx.x == 0) flag(a.status, i, kInval);
    return;
  }
  const int per_row = a.head_dim * a.size / 16;
  const long long pieces = static_cast<long long>(rows) * c.n_kv * per_row;
  char* const pool = side ? c.v : c.k;
  for (long long p0 = static_cast<long long>(part) * kCopyPieces; p0 < pieces; p0 += static_cast<long long>(parts) * kCopyPieces) {
    uint4 v[4];
    long long at[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const long long q = p0 + e * 256 + threadIdx.x;
      if (q < pieces) {
        const int row = static_cast<int>(q / per_row), ch = static_cast<int>(q - static_cast<long long>(row) * per_row);
        const int t = row / c.n_kv, h = row - t * c.n_kv;
        const long long o = (t * c.token_stride + h * c.head_stride) * a.size + ch * 16;
        v[e] = *reinterpret_cast<const uint4*>(pool + src * c.page_stride * a.size + o);
        at[e] = o;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const long long q = p0 + e * 256 + threadIdx.x;
      if (q < pieces) *reinterpret_cast<uint4*>(pool + dst * c.page_stride * a.size + at[e]) = v[e];
    }
  }
  if (a.size == 1 && part == 0) {
    float* const scales = side ? c.v_scale : c.k_scale;
    for (long long q = threadIdx.x; q < static_cast<long long>(rows) * c.n_kv; q += 256) {
      const int t = static_cast<int>(q / c.n_kv), h = static_cast<int>(q - static_cast<long long>(t) * c.n_kv);
      const long long o = t * c.s_token_stride + h * c.s_head_stride;
      scales[dst * c.s_page_stride + o] = scales[src * c.s_page_stride + o];
    }
  }
}

// ------------------------------------------------------------------ moving kept tokens together
// A thread owns 16 bytes of every position of a request (one side, head and piece; or one scale) and moves them in
// ascending order: keep[j] >= j, so a place is overwritten after it was read, by the same thread, and no other
// looks at it.  Eight positions' loads are in flight together (the stores of eight reach places below all later loads).
__global__ void __launch_bounds__(256) keep_kernel(const __grid_constant__ PagedKeepArgs a, const __grid_constant__ LayerPools l) {
  __shared__ long long from[kKeepMax], to[kKeepMax], sfrom[kKeepMax], sto[kKeepMax];
  const PagedCache& c = l.c[blockIdx.y];
  const int r = blockIdx.x, tid = threadIdx.x;
  const int b0 = __ldg(a.rq.begin + r), b1 = __ldg(a.rq.begin + r + 1), len = __ldg(a.rq.kv_len + r), kept = __ldg(a.n_keep + r);
  const int n = b1 - b0, base = len - n;
  const long long cap = static_cast<long long>(c.max_pages) * c.page_size;
  bool bad = !paged_request_ok(a.rq, b0, b1, len) || len > cap || base < 0 || kept < 0 || kept > n || kept > a.max_keep;
  const int32_t* const keep = a.keep + r * a.keep_stride;
  if (!bad && tid < kept) {
    const int k = __ldg(keep + tid);
    bad = k < 0 || k >= n || (tid > 0 && __ldg(keep + tid - 1) >= k);
  }
  const bool off = __syncthreads_or(bad);  // the request itself
  bad = false;
  if (!off && tid < kept) {
    const int32_t* const row = c.table + r * c.table_stride;
    const int s = base + __ldg(keep + tid), d = base + tid;
    bad = !paged_row(c, __ldg(row + s / c.page_size), s % c.page_size, 0, from + tid, sfrom + tid);
    bad |= !paged_row(c, __ldg(row + d / c.page_size), d % c.page_size, 0, to + tid, sto + tid);
  }
  bad = __syncthreads_or(bad) || off;
  if (tid == 0 && blockIdx.z == 0) {
    if (bad) flag(a.rq.status, r, kInval);
    if (a.kv_out && blockIdx.y == 0) a.kv_out[r] = off ? len : base + kept;
  }
  if (bad) return;
  const int per_row = a.head_dim * a.size / 16, cols = c.n_kv * per_row, column = blockIdx.z * 256 + tid;
  if (column < 2 * cols) {
    const int side = column >= cols, x = column - side * cols, h = x / per_row;
    char* const p = (side ? c.v : c.k) + h * c.head_stride * a.size + (x - h * per_row) * 16;
    for (int j0 = 0; j0 < kept; j0 += 8) {
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < kept) v[j] = *reinterpret_cast<const uint4*>(p + from[j0 + j] * a.size);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < kept && from[j0 + j] != to[j0 + j]) *reinterpret_cast<uint4*>(p + to[j0 + j] * a.size) = v[j];
    }
  } else if (a.size == 1 && column < 2 * cols + 2 * c.n_kv) {
    const int x = column - 2 * cols, side = x >= c.n_kv;
    float* const p = (side ? c.v_scale : c.k_scale) + (x - side * c.n_kv) * c.s_head_stride;
    for (int j0 = 0; j0 < kept; j0 += 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < kept) v[j] = p[sfrom[j0 + j]];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < kept) p[sto[j0 + j]] = v[j];
    }
  }
}

size_t resize_smem(int n_pages) {
  const size_t chunks = (static_cast<size_t>(n_pages) + kChunk - 1) / kChunk;
  return sizeof(ResizeShared) + chunks * 4 + (chunks + kCluster - 1) / kCluster * 128;
}

}  // namespace

cudaError_t launch_pages_resize(const PagesResizeArgs& a, cudaStream_t st) {
  static std::atomic<unsigned long long> done[2];
  cudaError_t e = set_smem_once(resize_kernel, static_cast<int>(resize_smem(1 << 22)), done[0]);
  if (e != cudaSuccess) return e;
  e = set_attr_once(resize_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, done[1]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kResizeThreads);
  cfg.dynamicSmemBytes = resize_smem(a.p.n_pages);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, resize_kernel, a);
}

cudaError_t launch_pages_fork(const PagesForkArgs& a, cudaStream_t st) {
  fork_kernel<<<a.n, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pages_copy(const PagesCopyArgs& a, const LayerPools& pools, int layers, cudaStream_t st) {
  const PagedCache& c = pools.c[0];
  const long long pieces = static_cast<long long>(c.page_size) * c.n_kv * (a.head_dim * a.size / 16);
  const int parts = static_cast<int>(std::min<long long>((pieces + kCopyPieces - 1) / kCopyPieces, 64));
  copy_kernel<<<dim3(static_cast<unsigned>(a.n) * 2 * parts, layers), 256, 0, st>>>(a, pools, parts);
  return cudaGetLastError();
}

cudaError_t launch_paged_keep(const PagedKeepArgs& a, const LayerPools& pools, int layers, cudaStream_t st) {
  const PagedCache& c = pools.c[0];
  const int columns = 2 * c.n_kv * (a.head_dim * a.size / 16) + (a.size == 1 ? 2 * c.n_kv : 0);
  keep_kernel<<<dim3(a.rq.n_req, layers, (columns + 255) / 256), 256, 0, st>>>(a, pools);
  return cudaGetLastError();
}

}  // namespace df2
