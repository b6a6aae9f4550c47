// Truncated sampling: temperature, top-k, top-p and min-p from the caller's uniforms.
//
// One thread-block cluster per row, each CTA a slice of it.  Every weight is a whole
// number, w = round(2^44 2^((x - max) log2(e) / T)), and sums of them are exact in 64 bits:
// no decision depends on the order in which the device adds, and equal logits get equal
// weights.  What stays is a prefix of the order (logit descending, id ascending), whose
// elements are the distinct 64-bit numbers (order-preserving key of the logit, ~id).  Two
// ways find its last element:
//  * The short one reads the row once.  Any CTA's k-th largest thread maximum is a lower
//    bound of the row's k-th largest logit (as is the least, over n CTAs, of their
//    k/n-th largest), and min_p bounds the logits outright; elements
//    above the bound known so far go to a list as the slice streams by (the bound is drawn
//    tighter after 1, 2, 4, ... chunks), and the `kept` row is filled with its cut value in
//    the same pass.  The first CTA sorts the few hundred candidates that pass the final
//    bound, reads top-k, top-p and min-p off the running weights, draws, and puts the logits that
//    stay into `kept`.  (top-p without top-k needs the weight of all: one more pass.)
//  * The long one, for rows whose nucleus is wide, or whose bound lets too many pass: a
//    histogram of counts (top-k) or weights (top-p) over the weight's exponent in steps of
//    1/32, whose bins spread the shared-memory atomics; the bin with the border is sorted as
//    above or, where equal logits flood it, searched by the digits of the 64-bit number.
//
// Measured with 248320 fp32 logits a row: 128 rows, top-k 50, the kept rows written (254 MB), 74 us; with mixed settings
// 127 to 189 us, by the rows with a wide nucleus among them (three passes over the row); one row
// 24 to 39 us, bound by latency (a 16-CTA cluster: 9 us of streaming, the rest barriers, the sort and the draw).
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "sample.h"

namespace cg = cooperative_groups;

namespace df2 {
namespace {

constexpr int kThreads = 512;   // (256, four CTAs to an SM: rows of one kind gain, long rows among short ones cost more)
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCtas = 16;
constexpr int kSlice = (1 << 17) - 8;  // most elements of a CTA (its histogram adds 15-bit pieces in 32 bits)
constexpr int kGroups = 2;       // groups of 4 consecutive elements a thread holds of a chunk
constexpr int kChunk = kThreads * 4 * kGroups;
constexpr int kList = 2048;      // candidates of a CTA
constexpr int kSort = 2048;      // candidates of a row
constexpr int kShortK = 384;     // largest top_k of the short way (of a CTA's 512 thread maxima)
constexpr int kProbe = 384;      // thread maxima above the CTAs' bounds, in all, for top-p alone
constexpr int kWaveCtas = 2;     // CTAs an SM holds
// The rows of a launch: all; those of the long way, where they are few; the others and, where they are many, those too.
enum Part { kAll, kFew, kRest };
constexpr float kCut = -1e30f;

// round(2^31 2^(j / 32))
__constant__ uint32_t kPow[32] = {
    2147483648u, 2194507417u, 2242560872u, 2291666561u, 2341847524u, 2393127307u, 2445529972u, 2499080105u,
    2553802834u, 2609723834u, 2666869345u, 2725266179u, 2784941738u, 2845924021u, 2908241642u, 2971923842u,
    3037000500u, 3103502151u, 3171459999u, 3240905930u, 3311872529u, 3384393094u, 3458501653u, 3534232978u,
    3611622603u, 3690706840u, 3771522796u, 3854108391u, 3938502376u, 4024744348u, 4112874773u, 4202935003u};

struct Scale {
  float xmax, ch, cl;  // log2(e) / T as ch + cl
};

template <int T>  // 0: bf16, 1: fp16, 2: fp32
DF2_DEV float load1(const char* p, int i) {
  // (+ 0 makes one zero of the two, which the order would otherwise tell apart)
  if constexpr (T == 2) return reinterpret_cast<const float*>(p)[i] + 0.f;
  const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
  if constexpr (T == 0) return bf16_to_f32(b) + 0.f;
  return __half2float(__ushort_as_half(b)) + 0.f;
}

// Elements i .. i + 3 of a row; vec: the row is aligned for one wide load.
template <int T>
DF2_DEV void load4(const char* p, int i, bool vec, float (&x)[4]) {
  if (!vec) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = load1<T>(p, i + e);
  } else if constexpr (T == 2) {
    const float4 v = *reinterpret_cast<const float4*>(p + 4ll * i);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p + 2ll * i);
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint16_t b = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
      x[e] = T == 0 ? bf16_to_f32(b) : __half2float(__ushort_as_half(b));
    }
  }
}

// 2^44 2^((x - xmax) (ch + cl)), rounded.  The exponent is carried as a sum of two floats (the
// difference's own rounding included); 2^(j / 32) comes from a 32-bit table and the rest, within
// 2^-6, from four terms of its series, applied as a 28-bit fraction: about 29 bits, with errors of either sign.
// Roundings to integers are sums with 1.5 * 2^23, and the table has a copy for each lane: conversions and bank
// conflicts bounded the passes over whole rows (`pw` is this lane's copy, entries 32 apart).
DF2_DEV unsigned long long weight(float x, const Scale& s, const uint32_t* pw) {
  constexpr float kMagic = 12582912.f;
  const float d = x - s.xmax;
  const float th = d * s.ch;
  if (!(th > -46.f)) return 0ull;
  const float bb = d - x;
  const float e = (x - (d - bb)) + (-s.xmax - bb);
  const float tl = fmaf(d, s.ch, -th) + fmaf(d, s.cl, e * s.ch);
  const float t = fmaf(th, 32.f, kMagic), nj = t - kMagic;
  const int n = __float_as_int(t) - __float_as_int(kMagic);
  const float r = fmaf(nj, -0.03125f, th) + tl;
  // 2^r - 1 = r ln 2 + (r ln 2)^2 / 2 + ...
  float q = fmaf(r, 0.0096181291f, 0.0555041087f);
  q = fmaf(q, r, 0.2402265070f);
  q = fmaf(q, r, 0.6931471806f);
  q *= r;
  const int qi = __float_as_int(fmaf(q, 268435456.f, kMagic)) - __float_as_int(kMagic);  // 2^28 q, within +- 2^22
  const uint32_t p = pw[(n & 31) * 32];
  const uint32_t m = p + static_cast<uint32_t>(__mulhi(static_cast<int>(p >> 1), qi << 5));
  const int up = 13 + (n >> 5);  // 2^31 of m is 2^44
  if (up >= 0) return static_cast<unsigned long long>(m) * (1u << up);
  return up < -31 ? 0ull : ((m >> (-up - 1)) + 1u) >> 1;
}

DF2_DEV unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The bin of the weight's exponent: -rint(32 log2 w), by the rounded difference's product alone, so it
// never falls where the logit falls; at most kBins - 1.
DF2_DEV uint32_t weight_step(float x, const Scale& s) {
  const float th = (x - s.xmax) * s.ch;
  return th > -46.f ? static_cast<uint32_t>(__float_as_int(fmaf(th, -32.f, 12582912.f)) - __float_as_int(12582912.f)) : kBins - 1;
}


struct Shared {
  union {
    unsigned long long hist[kBins];   // the digits' histogram
    uint32_t piece[3][kBins];         // the steps' histogram: 15-bit pieces of counts or weights
    unsigned long long sort[kSort];
  };
  union {
    unsigned long long list[kList];      // this CTA's candidates, until they are gathered
    unsigned long long w[kSort];         // weights of the sorted candidates; a histogram's sums
  };
  unsigned long long warp_sum[kWarps];   // of this CTA's warps
  unsigned long long scan[kWarps];
  unsigned long long best;               // this CTA's largest element
  unsigned long long total;
  unsigned long long before;             // weight or count above the digit found
  unsigned long long result;             // the last element that stays; 0: not found
  uint32_t tau, share, count, digit, bad, n_sort, run_max;
  uint32_t pw[32][32];  // the table, a copy for each lane
};

struct Ctx {
  cg::cluster_group cl;
  Shared* sh;
  int rank, ctas, lo, n;          // this CTA's ids [lo, lo + n)
  int wlo, whi;                   // this warp's part of them
};

// Exclusive sum over the block's threads, in thread order; the block's sum in `all`.
DF2_DEV unsigned long long block_scan(Shared* sh, unsigned long long v, unsigned long long& all) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh->scan[wid] = x;
  __syncthreads();
  unsigned long long base = 0;
  all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const unsigned long long t = sh->scan[i];
    if (i < wid) base += t;
    all += t;
  }
  __syncthreads();
  return base + x - v;
}

// This CTA's sum into `total` (each warp's in warp_sum); the caller synchronises the cluster.
DF2_DEV unsigned long long put_total(Ctx& c, unsigned long long mine) {
  mine = warp_sum_u64(mine);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if (lane == 0) c.sh->warp_sum[wid] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned long long t = 0;
    for (int i = 0; i < kWarps; ++i) t += c.sh->warp_sum[i];
    c.sh->total = t;
  }
  return mine;
}

// Adds the cluster's histograms and finds the bin, from kBins - 1 down, at which the running sum
// first reaches the target; also the sum above it.  The bin found is never empty.  Each CTA adds its share of
// the bins and the first one searches the sums.  (All CTAs adding all bins: 134 us with 16 of them.)
template <bool PIECES, typename F>
DF2_DEV void find_bin(Ctx& c, F reached, uint32_t& bin, unsigned long long& above) {
  constexpr int kPer = kBins / kThreads;
  Shared* sh = c.sh;
  const int share = kBins / c.ctas;  // (a power of two)
  c.cl.sync();
  for (int b = c.rank * share + threadIdx.x; b < (c.rank + 1) * share; b += kThreads) {
    unsigned long long h = 0;
#pragma unroll 4
    for (int r = 0; r < c.ctas; ++r) {
      const Shared* o = c.cl.map_shared_rank(sh, r);
      h += PIECES ? o->piece[0][b] + (static_cast<unsigned long long>(o->piece[1][b]) << 15) +
                        (static_cast<unsigned long long>(o->piece[2][b]) << 30)
                  : o->hist[b];
    }
    sh->w[b] = h;
  }
  c.cl.sync();
  if (c.rank == 0) {
    const int b0 = kBins - 1 - kPer * static_cast<int>(threadIdx.x);
    unsigned long long h[kPer], sum = 0, all;
#pragma unroll
    for (int i = 0; i < kPer; ++i) h[i] = c.cl.map_shared_rank(sh, (b0 - i) / share)->w[b0 - i];
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += h[i];
    unsigned long long s = block_scan(sh, sum, all);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (h[i] != 0 && !reached(s) && reached(s + h[i])) {
        sh->digit = b0 - i;
        sh->before = s;
      }
      s += h[i];
    }
  }
  c.cl.sync();
  const Shared* first = c.cl.map_shared_rank(sh, 0);
  bin = first->digit;
  above = first->before;
}

// Sorts the first n2 (a power of two) elements, largest first.
DF2_DEV void sort_desc(unsigned long long* v, int n2) {
  for (int size = 2; size <= n2; size <<= 1)
    for (int st = size >> 1; st > 0; st >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < n2 / 2; i += kThreads) {
        const int a = 2 * i - (i & (st - 1)), b = a + st;
        const unsigned long long x = v[a], y = v[b];
        if ((x < y) == ((a & size) == 0)) {
          v[a] = y;
          v[b] = x;
        }
      }
    }
  __syncthreads();
}


// Whether (x, id) comes no later than (lx, lid) in the order.
DF2_DEV bool reaches(float x, int id, float lx, int lid) { return x > lx || (x == lx && id <= lid); }

// Appends the warp's elements that are `in` to this CTA's list.
DF2_DEV void append(Shared* sh, bool in, unsigned long long v) {
  const uint32_t m = __ballot_sync(0xffffffffu, in);
  if (m == 0) return;
  const int lane = threadIdx.x & 31, lead = __ffs(m) - 1;
  uint32_t at = 0;
  if (lane == lead) at = atomicAdd(&sh->count, __popc(m));
  at = __shfl_sync(0xffffffffu, at, lead) + __popc(m & ((1u << lane) - 1u));
  if (in && at < kList) sh->list[at] = v;
}

// The first CTA gathers the cluster's lists (elements >= least) into its sort buffer, sorted; returns the number,
// or more than kSort if they do not fit.  Called by every thread of that CTA after a cluster barrier.
DF2_DEV int gather_sorted(Ctx& c, unsigned long long least) {
  Shared* sh = c.sh;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if (threadIdx.x == 0) sh->n_sort = 0;
  const uint32_t count = lane < c.ctas ? c.cl.map_shared_rank(sh, lane)->count : 0u;
  const bool over = __any_sync(0xffffffffu, count > kList);
  __syncthreads();
  // a warp for each list, or several where there are fewer lists than warps
  const int shares = c.ctas < kWarps ? kWarps / c.ctas : 1;
  for (int r = wid % c.ctas; !over && r < c.ctas; r += kWarps) {
    const int cr = static_cast<int>(__shfl_sync(0xffffffffu, count, r));
    const Shared* o = c.cl.map_shared_rank(sh, r);
    for (int i0 = (shares > 1 ? wid / c.ctas : 0) * 32; i0 < cr; i0 += shares * 32) {
      const unsigned long long v = i0 + lane < cr ? o->list[i0 + lane] : 0ull;
      const bool in = i0 + lane < cr && v >= least;
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      if (m == 0) continue;
      uint32_t at = 0;
      if (lane == 0) at = atomicAdd(&sh->n_sort, __popc(m));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1u));
      if (in && at < kSort) sh->sort[at] = v;
    }
  }
  __syncthreads();
  const int n = over ? kSort + 1 : static_cast<int>(sh->n_sort);
  if (n > kSort) return n;
  int n2 = 64;
  while (n2 < n) n2 <<= 1;
  for (int i = n + threadIdx.x; i < n2; i += kThreads) sh->sort[i] = 0;
  sort_desc(sh->sort, n2);
  return n;
}

template <int T>
DF2_DEV void sample_row(const SampleArgs& a, int part, int few) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Shared& shm = *reinterpret_cast<Shared*>(smem_raw);
  Ctx c{cg::this_cluster(), &shm};
  c.rank = c.cl.block_rank();
  c.ctas = c.cl.num_blocks();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int row = blockIdx.x / c.ctas;
  if (part != kAll) {  // the cluster's row among the part's (of every kThreads rows)
    const int width = part == kFew ? few : kThreads, place = row % width, r = row / width * kThreads + threadIdx.x;
    bool passes = false;
    if (r < a.n_rows) {
      const int k = a.top_k ? a.top_k[r] : 0;
      passes = a.temperature[r] > 0.f && (k <= 0 || k > kShortK) &&
               ((a.top_p && a.top_p[r] < 1.f) || k > 0 || !(a.min_p && a.min_p[r] > 0.f));
    }
    const int n_long = __syncthreads_count(passes);
    const bool many = n_long > few;
    // (many: the long ones first)
    const bool first = r < a.n_rows && (part == kFew ? passes && !many : passes == many);
    const bool second = r < a.n_rows && part == kRest && many && !passes;
    const uint32_t those = __ballot_sync(0xffffffffu, first);
    const uint32_t these = __ballot_sync(0xffffffffu, second);
    if (lane == 0) shm.warp_sum[wid] = __popc(those), shm.scan[wid] = __popc(these);
    __syncthreads();
    const uint32_t below = (1u << lane) - 1;
    int before = __popc(second ? these & below : those & below), all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int x = static_cast<int>(shm.warp_sum[w]), y = static_cast<int>(shm.scan[w]);
      before += w < wid ? (second ? y : x) : 0;
      before += second ? x : 0;
      all += x + y;
    }
    if (place >= all) return;  // (the whole cluster)
    if ((first || second) && before == place) shm.digit = r;
    __syncthreads();
    row = static_cast<int>(shm.digit);
  }
  const int per = ((a.vocab + c.ctas - 1) / c.ctas + 7) & ~7;
  c.lo = min(a.vocab, c.rank * per);
  c.n = min(a.vocab, c.lo + per) - c.lo;
  const int wper = ((c.n + kWarps - 1) / kWarps + 31) & ~31;
  c.wlo = min(c.n, wid * wper);
  c.whi = min(c.n, c.wlo + wper);
  const char* src = static_cast<const char*>(a.logits) + (row * a.row_stride + c.lo) * (T == 2 ? 4 : 2);
  const bool vec = (reinterpret_cast<uintptr_t>(src) & (T == 2 ? 15 : 7)) == 0;
  float* const kept = a.kept ? a.kept + row * a.kept_stride + c.lo : nullptr;
  const bool kvec = (reinterpret_cast<uintptr_t>(kept) & 15) == 0;
  const bool fill = kept && !a.kept_in_place;  // (in place the logits may be read again)
  auto element = [&](float x, int i) { return topk_key(x, c.lo + i); };
  for (int i = threadIdx.x; i < 32 * 32; i += kThreads) shm.pw[i >> 5][i & 31] = kPow[i >> 5];
  const uint32_t* const pw = &shm.pw[0][lane];
  if (threadIdx.x == 0) shm.bad = shm.count = shm.run_max = 0;
  const float temp = a.temperature[row], u = a.uniform[row];
  const float top_p = a.top_p ? a.top_p[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
  const int top_k_raw = a.top_k ? a.top_k[row] : 0;
  const int top_k = top_k_raw > 0 && top_k_raw < a.vocab ? top_k_raw : 0;
  const bool whole = a.vocab <= kList;  // every element is a candidate
  // thread maxima that the bound has to leave above it (0: no such bound)
  const int want = temp == 0.f || whole ? 0 : (top_k ? (top_k <= kShortK ? top_k : 0) : (top_p < 1.f ? max(16, kProbe / c.ctas) : 0));
  // min_p bounds the logits, x - max >= T ln(min_p), with room for every rounding here; but top-p
  // after top-k is a share of all that top-k left
  const bool by_min = !whole && temp > 0.f && min_p > 0.f && min_p <= 1.f && !(top_k && top_p < 1.f);
  const float reach = by_min ? temp * logf(min_p) * 1.0001f - 1e-4f * temp : 0.f;
  auto min_bound = [&](float x) { return float_order(x + (reach - 1e-6f * fabsf(x))); };
  const bool listing = temp > 0.f && (want != 0 || by_min || whole);
  __syncthreads();

  // ---- the slice streams by: each thread's largest, nonfinite ones, candidates
  unsigned long long best = 0;
  bool bad = false;
  uint32_t tau = 0;
  float best_x = -INFINITY;
  auto nth = [&](int nth_largest, int low) {  // a bound from below, down to bit `low`, of the thread maxima's n-th largest so far
    const uint32_t mine = static_cast<uint32_t>(best >> 32);
    uint32_t t0 = 0;
#pragma unroll 1
    for (int b = 31; b >= low; --b) {
      const uint32_t t = t0 | (1u << b);
      if (__syncthreads_count(mine >= t) >= nth_largest) t0 = t;
    }
    return t0;
  };
  auto tighten = [&](int low) { tau = max(tau, nth(want, low)); };
  const int chunks = (c.n + kChunk - 1) / kChunk;
  float next[kGroups][4];
  auto fetch = [&](int ck) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int i = ck * kChunk + threadIdx.x * 4 + g * kThreads * 4;
      if (i + 3 < c.n) {
        load4<T>(src, i, vec, next[g]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) next[g][e] = i + e < c.n ? load1<T>(src, i + e) : -INFINITY;
      }
    }
  };
  fetch(0);
  for (int ck = 0; ck < chunks; ++ck) {
    float x[kGroups][4];
    const int base = ck * kChunk + threadIdx.x * 4;
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[g][e] = next[g][e] + 0.f;  // (one zero, see load1; here, or the fetch would wait)
    fetch(ck + 1);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int i = base + g * kThreads * 4;
      bad |= !(x[g][0] < INFINITY && x[g][1] < INFINITY && x[g][2] < INFINITY && x[g][3] < INFINITY);  // NaN or +infinity
      const float m = fmaxf(fmaxf(x[g][0], x[g][1]), fmaxf(x[g][2], x[g][3]));
      if (i < c.n && (best == 0 || m > best_x)) {
        best_x = m;
#pragma unroll
        for (int e = 3; e >= 0; --e)  // (the smallest id of equal ones)
          if (i + e < c.n && x[g][e] == m) best = element(m, i + e);
      }
      if (fill) {
        if (kvec && i + 3 < c.n) {
          *reinterpret_cast<float4*>(kept + i) = make_float4(kCut, kCut, kCut, kCut);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < c.n) kept[i + e] = kCut;
        }
      }
    }
    if (listing) {
      if (by_min) {  // the bound of the largest logit so far
        const uint32_t wm = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(best >> 32));
        if (lane == 0) atomicMax(&shm.run_max, wm);
        __syncthreads();
        const float top = order_to_float(shm.run_max);
        if (top > -INFINITY && top < INFINITY) tau = max(tau, min_bound(top));
      }
      if (want && (ck & (ck + 1)) == 0) tighten(20);  // after 1, 2, 4, ... chunks
      const float tau_x = tau > 0x007FFFFFu ? order_to_float(tau) : -INFINITY;  // (every element from -infinity on)
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int i = base + g * kThreads * 4;
        const float m = fmaxf(fmaxf(x[g][0], x[g][1]), fmaxf(x[g][2], x[g][3]));
        if (m >= tau_x) {  // (a few in a hundred: no need to gather the warp's)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < c.n && x[g][e] >= tau_x) {
              const uint32_t at = atomicAdd(&shm.count, 1u);
              if (at < kList) shm.list[at] = element(x[g][e], i + e);
            }
        }
      }
    }
  }
  // at the end also the bound that all CTAs share: each has its part of top_k above its own bound, so the row has
  // top_k above the least of them
  uint32_t share = 0;
  if (want && chunks > 0) {
    tighten(18);
    if (top_k && c.ctas > 1) share = nth((top_k + c.ctas - 1) / c.ctas, 18);
  }
  best = warp_max_u64(best);
  if (lane == 0) shm.warp_sum[wid] = best;
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&shm.bad, 1u);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kWarps; ++i) best = shm.warp_sum[i] > best ? shm.warp_sum[i] : best;
    shm.best = best;
    shm.tau = tau;
    shm.share = share;
  }
  c.cl.sync();
  uint32_t any_bad = 0;
  best = 0;
  if (lane < c.ctas) {
    const Shared* o = c.cl.map_shared_rank(&shm, lane);
    any_bad = o->bad;
    best = o->best;
    tau = o->tau;
    share = o->share;
  } else {
    share = 0xFFFFFFFFu;
  }
  any_bad = __any_sync(0xffffffffu, any_bad != 0);
  best = warp_max_u64(best);
  tau = max(__reduce_max_sync(0xffffffffu, tau), __reduce_min_sync(0xffffffffu, share));
  Scale s;
  s.xmax = key_value(best);
  int status = 0;
  if (any_bad || !(s.xmax > -INFINITY)) status = 2;  // DFLASH2_E_NONFINITE
  if (!(temp >= 0.f) || !(temp < INFINITY) || !(top_p > 0.f) || !(min_p >= 0.f) || !(min_p <= 1.f) || !(u >= 0.f) || !(u < 1.f))
    status = 1;  // DFLASH2_E_INVAL
  if (status != 0 || temp == 0.f) {
    const int id = static_cast<int>(key_index(best)) - c.lo;
    if (kept)
      for (int i = threadIdx.x; i < c.n; i += kThreads) {
        const bool stays = status == 0 && i == id;
        if (!fill || stays) kept[i] = stays ? s.xmax : kCut;
      }
    if (c.rank == 0 && threadIdx.x == 0) {
      a.token[row] = status ? -1 : id + c.lo;
      if (a.prob) a.prob[row] = status ? 0.f : 1.f;
      if (a.status) a.status[row] = status;
    }
    c.cl.sync();  // (another CTA may still read this one's shared memory)
    return;
  }
  {
    const double cc = 1.4426950408889634 / static_cast<double>(temp);
    s.ch = static_cast<float>(cc);
    s.cl = static_cast<float>(cc - static_cast<double>(s.ch));
    if (!(s.ch < INFINITY)) s.ch = 3.4028235e38f, s.cl = 0.f;
  }
  // (compared as whole numbers: conversions to 64-bit floats, two a clock, bounded the passes over whole rows)
  const unsigned long long floor_w = static_cast<unsigned long long>(ceil(static_cast<double>(min_p) * 17592186044416.0));  // 2^44
  bool bounded = whole || (top_k != 0 && want != 0);  // every element that may stay is a candidate
  if (by_min) {
    const uint32_t t = min_bound(s.xmax);
    if (t >= tau) {
      tau = t;
      bounded = true;
    }
  }

  // Adds the weight (or 1) of every element >= least to the steps' histogram; returns the thread's sum.
  auto steps = [&](bool by_weight, unsigned long long least) {
    const float least_x = least ? key_value(least) : -INFINITY;
    const int least_id = least ? static_cast<int>(key_index(least)) : a.vocab;
    for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&shm.piece[0][0])[i] = 0;
    __syncthreads();
    unsigned long long z = 0;
    for (int i0 = threadIdx.x; i0 < c.n; i0 += 8 * kThreads) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = i0 + e * kThreads < c.n ? load1<T>(src, i0 + e * kThreads) : -INFINITY;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = i0 + e * kThreads;
        if (i >= c.n || !reaches(x[e], c.lo + i, least_x, least_id)) continue;
        const unsigned long long w = by_weight ? weight(x[e], s, pw) : 1ull;
        if (w == 0) continue;
        z += w;
        const int b = kBins - 1 - weight_step(x[e], s);
        atomicAdd(&shm.piece[0][b], static_cast<uint32_t>(w) & 0x7FFFu);
        if (w >> 15) {
          atomicAdd(&shm.piece[1][b], static_cast<uint32_t>(w >> 15) & 0x7FFFu);
          if (w >> 30) atomicAdd(&shm.piece[2][b], static_cast<uint32_t>(w >> 30));
        }
      }
    }
    return z;
  };

  // ---- the short way
  double target = 0.0;   // top-p's share of the weight that top-k left
  bool have_steps = false;
  if (listing) {
    if (top_p < 1.f && top_k == 0) {
      put_total(c, steps(true, 0ull));
      have_steps = true;
      c.cl.sync();
      unsigned long long zt = 0;
      if (lane < c.ctas) zt = c.cl.map_shared_rank(&shm, lane)->total;
      target = static_cast<double>(top_p) * static_cast<double>(warp_sum_u64(zt));
    }
    // (the first CTA's sort buffer shares the histogram's memory, which waits in registers meanwhile)
    unsigned long long* const pieces = reinterpret_cast<unsigned long long*>(&shm.piece[0][0]);
    unsigned long long save[3 * kBins / 2 / kThreads];
    if (c.rank == 0) {
      if (have_steps) {
#pragma unroll
        for (int i = 0; i < 3 * kBins / 2 / kThreads; ++i) save[i] = pieces[threadIdx.x + i * kThreads];
        __syncthreads();
      }
      const int n = gather_sorted(c, static_cast<unsigned long long>(tau) << 32);
      unsigned long long result = 0;
      if (n <= kSort) {
        constexpr int kPer = kSort / kThreads;
        const int lim = top_k ? min(top_k, n) : n;
        unsigned long long w[kPer], sum_w = 0, all;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int j = threadIdx.x * kPer + i;
          w[i] = j < lim ? weight(key_value(shm.sort[j]), s, pw) : 0ull;
          sum_w += w[i];
          shm.w[j] = w[i];
        }
        unsigned long long run = block_scan(&shm, sum_w, all);
        const double goal_w = top_k ? static_cast<double>(top_p) * static_cast<double>(all) : target;
        int stay = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int j = threadIdx.x * kPer + i;
          if (j < lim && (j == 0 || top_p >= 1.f || static_cast<double>(run) < goal_w) && w[i] >= floor_w &&
              (shm.sort[j] >> 32) > 0x007FFFFFu)  // (above -infinity)
            ++stay;
          run += w[i];
        }
        unsigned long long total, kk;
        block_scan(&shm, static_cast<unsigned long long>(stay), kk);
        const int K = static_cast<int>(kk);  // a prefix stays
        if (bounded || K < n || n == a.vocab) {
          result = shm.sort[K - 1];
          sum_w = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i) sum_w += static_cast<int>(threadIdx.x) * kPer + i < K ? w[i] : 0ull;
          block_scan(&shm, sum_w, total);
          const double goal = static_cast<double>(u) * static_cast<double>(total);
          // the draw in id order: the weight of the smaller ids among those that stay
          for (int j = threadIdx.x; j < K; j += kThreads) {
            const unsigned long long v = shm.sort[j];
            const uint32_t me = static_cast<uint32_t>(v);  // ~id: larger for smaller ids
            unsigned long long before = 0;
#pragma unroll 4
            for (int i = 0; i < K; ++i) before += static_cast<uint32_t>(shm.sort[i]) > me ? shm.w[i] : 0ull;
            const unsigned long long wj = shm.w[j];
            const int id = static_cast<int>(0xFFFFFFFFu - me);
            if (static_cast<double>(before) <= goal && static_cast<double>(before + wj) > goal) {
              a.token[row] = id;
              if (a.prob) a.prob[row] = static_cast<float>(static_cast<double>(wj) / static_cast<double>(total));
              if (a.status) a.status[row] = 0;
            }
            if (fill) kept[id] = key_value(v);  // (every CTA's filling came before the barrier; rank 0's row starts at id 0)
          }
        }
      }
      __syncthreads();
      if (threadIdx.x == 0) shm.result = result;
      if (have_steps && result == 0) {
#pragma unroll
        for (int i = 0; i < 3 * kBins / 2 / kThreads; ++i) pieces[threadIdx.x + i * kThreads] = save[i];
      }
    }
    c.cl.sync();
    const unsigned long long last = c.cl.map_shared_rank(&shm, 0)->result;
    c.cl.sync();
    if (last != 0) {
      if (kept && !fill)
        for (int i = threadIdx.x; i < c.n; i += kThreads) {
          const float x = load1<T>(src, i);
          kept[i] = element(x, i) >= last ? x : kCut;
        }
      return;
    }
  }

  // ---- the long way
  unsigned long long least = 0;  // elements >= it stay
  for (int stage = 0; stage < 2; ++stage) {  // 0: top-k (counts), 1: top-p (weights)
    const bool by_weight = stage == 1;
    if (!by_weight && top_k == 0) continue;
    if (by_weight && !(top_p < 1.f)) continue;
    if (!(by_weight && have_steps)) {
      put_total(c, steps(by_weight, least));
      c.cl.sync();
      if (by_weight) {
        unsigned long long zt = 0;
        if (lane < c.ctas) zt = c.cl.map_shared_rank(&shm, lane)->total;
        target = static_cast<double>(top_p) * static_cast<double>(warp_sum_u64(zt));
      }
    }
    const unsigned long long want_k = static_cast<unsigned long long>(top_k);
    unsigned long long above = 0;
    auto reached = [&](unsigned long long v) {
      return by_weight ? static_cast<double>(above + v) >= target : above + v >= want_k;
    };
    auto value = [&](float x) { return by_weight ? weight(x, s, pw) : 1ull; };
    uint32_t bin;
    unsigned long long up;
    if (threadIdx.x == 0) shm.count = 0;
    find_bin<true>(c, reached, bin, up);
    above = up;
    const uint32_t step = kBins - 1 - bin;
    // the bin's elements to the lists
    for (int i0 = 0; i0 < c.n; i0 += 8 * kThreads) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = i0 + e * kThreads + threadIdx.x;
        x[e] = i < c.n ? load1<T>(src, i) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = i0 + e * kThreads + threadIdx.x;
        const unsigned long long v = element(x[e], i);
        append(&shm, i < c.n && v >= least && weight_step(x[e], s) == step, v);
      }
    }
    c.cl.sync();
    if (c.rank == 0) {
      const int n = gather_sorted(c, 0ull);
      if (threadIdx.x == 0) shm.result = 0;
      __syncthreads();
      if (n <= kSort) {
        constexpr int kPer = kSort / kThreads;
        unsigned long long w[kPer], sum = 0, all;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int j = threadIdx.x * kPer + i;
          w[i] = j < n ? value(key_value(shm.sort[j])) : 0ull;
          sum += w[i];
        }
        unsigned long long run = block_scan(&shm, sum, all);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (w[i] != 0 && !reached(run) && reached(run + w[i])) shm.result = shm.sort[threadIdx.x * kPer + i];
          run += w[i];
        }
      }
    }
    c.cl.sync();
    unsigned long long last = c.cl.map_shared_rank(&shm, 0)->result;
    c.cl.sync();
    if (last == 0) {
      // equal logits flood the bin: its elements by the digits of (key, ~id): 11 + 11 + 10 and 11 + 8 bits
      // (ids are below 2^19)
      unsigned long long prefix = 0;
      int shift = 51;
      for (int round = 0; round < 5; ++round) {
        const int bits = round == 2 ? 10 : (round == 4 ? 8 : 11);
        shift -= bits;
        for (int i = threadIdx.x; i < kBins; i += kThreads) shm.hist[i] = 0;
        __syncthreads();
        for (int i0 = c.wlo; i0 < c.whi; i0 += 32) {
          const int i = i0 + lane;
          const float x = i < c.whi ? load1<T>(src, i) : 0.f;
          const unsigned long long v = element(x, i), e = ((v >> 32) << 19) | (v & 0x7FFFFu);
          const bool in = i < c.whi && v >= least && weight_step(x, s) == step && (round == 0 || (e >> (shift + bits)) == prefix);
          const uint32_t m = __ballot_sync(0xffffffffu, in);
          if (m == 0) continue;
          const uint32_t d = static_cast<uint32_t>(e >> shift) & ((1u << bits) - 1u);
          const unsigned long long w = in ? value(x) : 0ull;
          const uint32_t lead = __shfl_sync(0xffffffffu, d, __ffs(m) - 1);
          if (__all_sync(0xffffffffu, !in || d == lead)) {
            const unsigned long long t = warp_sum_u64(w);  // one digit for the warp
            if (lane == __ffs(m) - 1) atomicAdd(&shm.hist[d], t);
          } else if (in) {
            atomicAdd(&shm.hist[d], w);
          }
        }
        uint32_t digit;
        find_bin<false>(c, reached, digit, up);
        above += up;
        prefix = (prefix << bits) | digit;
      }
      last = ((prefix >> 19) << 32) | (0xFFF80000u | (prefix & 0x7FFFFu));
    }
    least = last;
    have_steps = false;
  }

  // ---- the weight left, and the draw
  const float least_x = least ? key_value(least) : -INFINITY;
  const int least_id = least ? static_cast<int>(key_index(least)) : a.vocab;
  auto left = [&](int i, float x, bool& stays) -> unsigned long long {
    stays = x > -INFINITY && reaches(x, c.lo + i, least_x, least_id);
    if (!stays) return 0ull;
    const unsigned long long w = weight(x, s, pw);
    stays = w >= floor_w;  // (a weight of zero may stay: it is then never drawn)
    return stays ? w : 0ull;
  };
  // In place, a cut logit is then no longer what it was: which ones stay is noted, a bit each.
  const bool noted = kept && !fill;
  uint32_t* const stay_bits = &shm.piece[0][0];
  static_assert(sizeof(shm.piece) * 8 >= kSlice, "a bit for every element of a slice");
  unsigned long long mine = 0;
  if (!noted) {
    for (int i0 = c.wlo + lane; i0 < c.whi; i0 += 256) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = i0 + 32 * e < c.whi ? load1<T>(src, i0 + 32 * e) : -INFINITY;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        bool stays;
        mine += left(i0 + 32 * e, x[e], stays);
        if (kept && i0 + 32 * e < c.whi) kept[i0 + 32 * e] = stays ? x[e] : kCut;
      }
    }
  } else {
#pragma unroll 1
    for (int b0 = c.wlo; b0 < c.whi; b0 += 32) {
      const int i = b0 + lane;
      const float x = i < c.whi ? load1<T>(src, i) : -INFINITY;
      bool stays;
      mine += left(i, x, stays);
      if (i < c.whi) kept[i] = stays ? x : kCut;
      const uint32_t m = __ballot_sync(0xffffffffu, stays);
      if (lane == 0) stay_bits[b0 >> 5] = m;
    }
  }
  auto again = [&](int i) -> unsigned long long {
    const float x = load1<T>(src, i);
    if (noted) return (stay_bits[i >> 5] >> (i & 31)) & 1u ? weight(x, s, pw) : 0ull;
    bool stays;
    return left(i, x, stays);
  };
  mine = put_total(c, mine);
  c.cl.sync();
  unsigned long long total = 0, before = 0;
  for (int r = 0; r < c.ctas; ++r) {
    const unsigned long long t = c.cl.map_shared_rank(&shm, r)->total;
    if (r < c.rank) before += t;
    total += t;
  }
  const double goal = static_cast<double>(u) * static_cast<double>(total);
  // the first id whose running weight exceeds the goal; u < 1, so there is one: the CTA that holds it, its warp's part of
  // the slice, then that part again, spread over the CTA's threads
  auto holds = [&](unsigned long long from, unsigned long long w) {
    return static_cast<double>(from) <= goal && static_cast<double>(from + w) > goal;
  };
  if (holds(before, shm.total)) {
    unsigned long long from = before;
    for (int i = 0; i < wid; ++i) from += shm.warp_sum[i];
    if (lane == 0 && holds(from, mine)) {
      shm.digit = static_cast<uint32_t>(wid);
      shm.before = from;
    }
    __syncthreads();
    const int lo = min(c.n, static_cast<int>(shm.digit) * wper), hi = min(c.n, lo + wper);
    const int each = (wper + kThreads - 1) / kThreads, i0 = lo + threadIdx.x * each;
    unsigned long long part = 0, all;
    for (int e = 0; e < each; ++e)
      if (i0 + e < hi) part += again(i0 + e);
    from = shm.before + block_scan(&shm, part, all);
    if (holds(from, part)) {
      for (int e = 0; e < each && i0 + e < hi; ++e) {
        const unsigned long long w = again(i0 + e);
        if (holds(from, w)) {
          a.token[row] = c.lo + i0 + e;
          if (a.prob) a.prob[row] = static_cast<float>(static_cast<double>(w) / static_cast<double>(total));
          if (a.status) a.status[row] = 0;
          break;
        }
        from += w;
      }
    }
  }
  c.cl.sync();
}

template <int T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, int part, int few) {
  if (part == kFew) pdl_trigger();
  sample_row<T>(a, part, few);
  // (begun while the launch before runs: one CTA waits for that one's end, so that what follows waits for both)
  if (part == kRest && blockIdx.x == 0) pdl_wait();
}

template <int T>
cudaError_t launch(const SampleArgs& a, int rows, int ctas, int part, int few, cudaStream_t st) {
  static std::atomic<unsigned long long> done[2];
  cudaError_t e = set_smem_once(sample_kernel<T>, sizeof(Shared), done[0]);
  if (e != cudaSuccess) return e;
  e = set_attr_once(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, done[1]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = part == kRest ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, part, few);
}

template <int T>
cudaError_t launch_rows(const SampleArgs& a, cudaStream_t st) {
  // CTAs per row: slices of at most kSlice elements; more while the GPU holds all rows' CTAs at a time and a slice
  // is more than 8192 elements.
  int ctas = 1;
  while ((a.vocab + ctas - 1) / ctas > kSlice - 8) ctas *= 2;
  while (ctas < kMaxCtas && a.n_rows * ctas * 2 <= kWaveCtas * a.num_sms && a.vocab / ctas > 8192) ctas *= 2;
  if (ctas == kMaxCtas || a.vocab / ctas <= 16384) return launch<T>(a, a.n_rows, ctas, kAll, 0, st);
  // The rows of the long way set the call's time: where they are few (half the rows at most, and
  // two and a half times what the GPU holds at once; of every kThreads rows) they begin first, with larger clusters; the others, for whom a large cluster only means more barriers, run
  // beside them.  The device knows which rows they are: clusters without a row end at once.
  // Measured (us), 248320 fp32 logits, clusters of four in one launch of two waves / this: 128 rows of mixed settings
  // 181 / 149, all top-k 95 / 74, all top-p 394 / 378; 32 rows 98 / 78, 87 / 43, 210 / 134; 512 rows 455 / 367, 242 / 250,
  // 1257 / 1261.  The same small clusters in one launch / this (another batch's settings; mixed, top-k, top-p): 128 rows of
  // 248320 258 / 129, 71 / 75, 367 / 377, in bf16 270 / 152, 88 / 92, 374 / 384; 32 rows 101 / 83, 41 / 45, 132 / 137; 128
  // rows of 131072 166 / 99, 52 / 56, 216 / 221; of 70000 101 / 71, 40 / 44, 134 / 139.
  const int most = ctas < 4 ? 8 : 2 * ctas, groups = (a.n_rows + kThreads - 1) / kThreads;
  const int few = std::max(1, std::min({5 * a.num_sms / most, a.n_rows / 2, kThreads}));
  const cudaError_t e = launch<T>(a, groups * (a.n_rows < few ? a.n_rows : few), most, kFew, few, st);
  return e != cudaSuccess ? e : launch<T>(a, a.n_rows, ctas, kRest, few, st);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st) {
  if (a.type == 0) return launch_rows<0>(a, st);
  return a.type == 1 ? launch_rows<1>(a, st) : launch_rows<2>(a, st);
}

}  // namespace df2
