// Truncated sampling: temperature, top-k, top-p and min-p from the caller's uniforms.
//
// One thread-block cluster per row; its CTAs keep the row's logits in shared memory, so
// HBM is read once.  Every weight is a whole number, w = round(2^44 2^((x - max) log2(e) / T)),
// and sums of them are exact in 64 bits: no decision depends on the order in which the
// device adds, and equal logits get equal weights.
//
// What stays is a threshold in the order (logit descending, id ascending).  It is found by
// radix selection on the logits' order-preserving 32-bit keys, 11 + 11 + 10 bits: counts for
// top-k, then weights for top-p (a digit's histogram lies in shared memory, one per CTA,
// and is added up through distributed shared memory).  Only elements that share the digits
// found so far enter the next histogram.  Of the elements that equal the threshold the
// ones with the smallest ids stay, as many as the count or the weight asks for.
#include <cooperative_groups.h>

#include "common.cuh"
#include "sample.h"

namespace cg = cooperative_groups;

namespace df2 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCtas = 8;
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

DF2_DEV float to_f32(const void* p, long long i, int type) {
  if (type == 2) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  if (type == 0) return bf16_to_f32(b);
  return __half2float(__ushort_as_half(b));
}

// 2^44 2^((x - xmax) (ch + cl)), rounded.  The exponent is carried as a sum of two floats (the
// difference's own rounding included); 2^(j / 32) comes from a 32-bit table and the rest, within
// 2^-6, from four terms of its series: about 30 bits, with errors of either sign.
DF2_DEV unsigned long long weight(float x, const Scale& s, const uint32_t* pw) {
  const float d = x - s.xmax;
  const float th = d * s.ch;
  if (!(th > -46.f)) return 0ull;
  const float bb = d - x;
  const float e = (x - (d - bb)) + (-s.xmax - bb);
  const float tl = fmaf(d, s.ch, -th) + fmaf(d, s.cl, e * s.ch);
  const float nj = rintf(th * 32.f);
  const float r = fmaf(nj, -0.03125f, th) + tl;
  // 2^r - 1 = r ln 2 + (r ln 2)^2 / 2 + ...
  float q = fmaf(r, 0.0096181291f, 0.0555041087f);
  q = fmaf(q, r, 0.2402265070f);
  q = fmaf(q, r, 0.6931471806f);
  q *= r;
  const int n = static_cast<int>(nj);
  const uint32_t p = pw[n & 31];
  const uint32_t m = p + static_cast<uint32_t>(__float2int_rn(static_cast<float>(p) * q));
  const int sh = -(n >> 5);
  const unsigned long long w = static_cast<unsigned long long>(m) << 13;
  return sh <= 0 ? w << -sh : (sh > 45 ? 0ull : (w + (1ull << (sh - 1))) >> sh);
}

DF2_DEV unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Shared {
  unsigned long long hist[kBins];
  unsigned long long warp_sum[kWarps];   // of this CTA's warps
  unsigned long long scan[kWarps + 1];
  unsigned long long best;               // (key << 32 | ~id) of this CTA
  unsigned long long total;
  unsigned long long before;             // weight or count above the digit found
  uint32_t digit, bad;
  uint32_t pw[32];
  int found;
};

struct Ctx {
  cg::cluster_group cl;
  Shared* sh;
  int rank, ctas, lo, n;          // this CTA's ids [lo, lo + n)
  int wlo, whi;                   // this warp's part of them
};

// Sum over the cluster of each CTA's `total`.
DF2_DEV unsigned long long cluster_total(Ctx& c, unsigned long long mine) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  mine = warp_sum_u64(mine);
  if (lane == 0) c.sh->warp_sum[wid] = mine;
  __syncthreads();
  if (wid == 0) {
    const unsigned long long t = warp_sum_u64(c.sh->warp_sum[lane]);
    if (lane == 0) c.sh->total = t;
  }
  c.cl.sync();
  unsigned long long t = 0;
  for (int r = 0; r < c.ctas; ++r) t += c.cl.map_shared_rank(c.sh, r)->total;
  c.cl.sync();
  return t;
}

// Adds the cluster's histograms and finds the digit, from the highest down, at which the
// running sum passes `target` (the first digit with sum above > = target - own); sets digit
// and the sum above it.  The digit found is never empty.
template <typename F>
DF2_DEV void find_digit(Ctx& c, F reached, uint32_t& digit, unsigned long long& above) {
  Shared* sh = c.sh;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  c.cl.sync();
  // thread t holds bins kBins - 1 - 2 t and kBins - 2 - 2 t (from the highest down)
  const int b0 = kBins - 1 - 2 * static_cast<int>(threadIdx.x), b1 = b0 - 1;
  unsigned long long h0 = 0, h1 = 0;
  for (int r = 0; r < c.ctas; ++r) {
    const Shared* o = c.cl.map_shared_rank(sh, r);
    h0 += o->hist[b0];
    h1 += o->hist[b1];
  }
  unsigned long long x = h0 + h1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh->scan[wid] = x;
  if (threadIdx.x == 0) sh->found = 0;
  __syncthreads();
  unsigned long long base = 0;
  for (int i = 0; i < wid; ++i) base += sh->scan[i];
  const unsigned long long s0 = base + x - h0 - h1;  // above b0
  // the digit: the sum above it has not reached the target, the sum with it has
  if (h0 != 0 && !reached(s0) && reached(s0 + h0)) {
    sh->digit = b0;
    sh->before = s0;
    sh->found = 1;
  }
  if (h1 != 0 && !reached(s0 + h0) && reached(s0 + h0 + h1)) {
    sh->digit = b1;
    sh->before = s0 + h0;
    sh->found = 1;
  }
  __syncthreads();
  digit = sh->digit;
  above = sh->before;
  c.cl.sync();
}

template <bool HELD>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ Shared shm;
  extern __shared__ float held[];
  Ctx c{cg::this_cluster(), &shm};
  c.rank = c.cl.block_rank();
  c.ctas = c.cl.num_blocks();
  const int row = blockIdx.x / c.ctas;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int per = (a.vocab + c.ctas - 1) / c.ctas;
  c.lo = min(a.vocab, c.rank * per);
  c.n = min(a.vocab, c.lo + per) - c.lo;
  const int wper = (c.n + kWarps - 1) / kWarps;
  c.wlo = min(c.n, wid * wper);
  c.whi = min(c.n, c.wlo + wper);
  const char* src = static_cast<const char*>(a.logits) + row * a.row_stride * (a.type == 2 ? 4 : 2);
  auto get = [&](int i) { return HELD ? held[i] : to_f32(src, c.lo + i, a.type); };
  if (threadIdx.x < 32) shm.pw[threadIdx.x] = kPow[threadIdx.x];
  if (threadIdx.x == 0) shm.bad = 0;
  __syncthreads();

  // ---- the largest logit, and nonfinite ones
  unsigned long long best = 0;
  bool bad = false;
  for (int i = c.wlo + lane; i < c.whi; i += 32) {
    const float x = to_f32(src, c.lo + i, a.type);
    if (HELD) held[i] = x;
    bad |= !(x < INFINITY);  // NaN or +infinity
    const unsigned long long k = topk_key(x, c.lo + i);
    best = k > best ? k : best;
  }
  best = warp_max_u64(best);
  if (lane == 0) shm.warp_sum[wid] = best;
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&shm.bad, 1u);
  __syncthreads();
  if (wid == 0) {
    const unsigned long long b = warp_max_u64(shm.warp_sum[lane]);
    if (lane == 0) shm.best = b;
  }
  c.cl.sync();
  uint32_t any_bad = 0;
  best = 0;
  for (int r = 0; r < c.ctas; ++r) {
    const Shared* o = c.cl.map_shared_rank(&shm, r);
    any_bad |= o->bad;
    best = o->best > best ? o->best : best;
  }
  const float temp = a.temperature[row], u = a.uniform[row];
  const float top_p = a.top_p ? a.top_p[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  Scale s;
  s.xmax = key_value(best);
  int status = 0;
  if (any_bad || !(s.xmax > -INFINITY)) status = 2;  // DFLASH2_E_NONFINITE
  if (!(temp >= 0.f) || !(temp < INFINITY) || !(top_p > 0.f) || !(min_p >= 0.f) || !(min_p <= 1.f) || !(u >= 0.f) || !(u < 1.f))
    status = 1;  // DFLASH2_E_INVAL
  float* const kept = a.kept ? a.kept + row * a.kept_stride : nullptr;
  if (status != 0 || temp == 0.f) {
    const int id = static_cast<int>(key_index(best));
    if (kept)
      for (int i = c.wlo + lane; i < c.whi; i += 32)
        kept[c.lo + i] = status == 0 && c.lo + i == id ? s.xmax : kCut;
    if (c.rank == 0 && threadIdx.x == 0) {
      a.token[row] = status ? -1 : id;
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

  // ---- the threshold: elements with a larger key stay, and `ties` of those that equal it
  uint32_t key_min = 0;                     // every key >= it is a candidate
  unsigned long long ties = ~0ull;          // of the elements with key == key_min, in id order
  bool cut = false;
  for (int stage = 0; stage < 2; ++stage) {  // 0: top-k (counts), 1: top-p (weights)
    const bool by_weight = stage == 1;
    if (!by_weight && !(top_k > 0 && top_k < a.vocab)) continue;
    if (by_weight && !(top_p < 1.f)) continue;
    // candidates of this stage: keys above key_min0, and the first ties0 that equal it.  Their weights
    // are equal, so which of the equal ones they are does not matter to the sums below.
    const uint32_t key0 = key_min;
    const unsigned long long ties0 = ties;
    double target = 0.0;
    if (by_weight) {
      unsigned long long z = 0;
      for (int i = c.wlo + lane; i < c.whi; i += 32) {
        const float x = get(i);
        const uint32_t k = float_order(x);
        if (k > key0 || (k == key0 && ties0 == ~0ull)) z += weight(x, s, shm.pw);
      }
      z = cluster_total(c, z);
      if (ties0 != ~0ull) z += ties0 * weight(order_to_float(key0), s, shm.pw);
      target = static_cast<double>(top_p) * static_cast<double>(z);
    }
    unsigned long long above = 0;
    uint32_t prefix = 0;
    int shift = 21, bits = 11;
    for (int round = 0; round < 3; ++round) {
      for (int i = threadIdx.x; i < kBins; i += kThreads) shm.hist[i] = 0;
      __syncthreads();
      for (int i = c.wlo + lane; i < c.whi; i += 32) {
        const float x = get(i);
        const uint32_t k = float_order(x);
        if (k < key0 || (round > 0 && (k >> (shift + bits)) != prefix)) continue;
        if (by_weight && k == key0 && ties0 != ~0ull) continue;  // added once below
        atomicAdd(&shm.hist[(k >> shift) & (kBins - 1)], by_weight ? weight(x, s, shm.pw) : 1ull);
      }
      __syncthreads();
      if (by_weight && ties0 != ~0ull && c.rank == 0 && threadIdx.x == 0 &&
          (round == 0 || (key0 >> (shift + bits)) == prefix))
        shm.hist[(key0 >> shift) & (kBins - 1)] += ties0 * weight(order_to_float(key0), s, shm.pw);
      uint32_t digit;
      unsigned long long up;
      const unsigned long long already = above;
      if (by_weight) {
        find_digit(c, [&](unsigned long long v) { return static_cast<double>(already + v) >= target; }, digit, up);
      } else {
        const unsigned long long want = static_cast<unsigned long long>(top_k);
        find_digit(c, [&](unsigned long long v) { return already + v >= want; }, digit, up);
      }
      above += up;
      prefix = round == 0 ? digit : (prefix << bits) | digit;
      if (round == 0) shift = 10;
      else if (round == 1) shift = 0, bits = 10;
    }
    key_min = prefix;
    cut = true;
    if (by_weight) {
      const unsigned long long w = weight(order_to_float(key_min), s, shm.pw);
      // the j-th equal element stays while above + j w < target
      unsigned long long r = 1;
      if (w != 0) {
        const double left = (target - static_cast<double>(above)) / static_cast<double>(w);
        r = static_cast<unsigned long long>(left);
        while (r > 0 && static_cast<double>(above + (r - 1) * w) >= target) --r;
        while (static_cast<double>(above + r * w) < target) ++r;
        if (r == 0) r = 1;
      }
      ties = (key_min == key0 && ties0 < r) ? ties0 : r;
    } else {
      ties = static_cast<unsigned long long>(top_k) - above;
    }
  }

  // ---- of the equal elements the first `ties` stay: the id of the last one
  int last_id = a.vocab;
  if (cut) {
    unsigned long long eq = 0;
    for (int i = c.wlo + lane; i < c.whi; i += 32) eq += float_order(get(i)) == key_min ? 1 : 0;
    eq = warp_sum_u64(eq);
    if (lane == 0) shm.warp_sum[wid] = eq;
    __syncthreads();
    if (wid == 0) {
      const unsigned long long t = warp_sum_u64(shm.warp_sum[lane]);
      if (lane == 0) shm.total = t;
    }
    if (threadIdx.x == 0) shm.found = -1;
    c.cl.sync();
    unsigned long long before = 0;
    for (int r = 0; r < c.rank; ++r) before += c.cl.map_shared_rank(&shm, r)->total;
    for (int i = 0; i < wid; ++i) before += shm.warp_sum[i];
    if (before < ties && before + eq >= ties) {  // this warp holds the last one that stays
      for (int i0 = c.wlo; i0 < c.whi; i0 += 32) {
        const int i = i0 + lane;
        const bool hit = i < c.whi && float_order(get(i)) == key_min;
        const uint32_t m = __ballot_sync(0xffffffffu, hit);
        const int cnt = __popc(m);
        if (before + cnt >= ties) {
          const int need = static_cast<int>(ties - before);  // 1-based
          if (hit && __popc(m & ((2u << lane) - 1u)) == need) shm.found = c.lo + i;
          break;
        }
        before += cnt;
      }
    }
    c.cl.sync();
    for (int r = 0; r < c.ctas; ++r) {
      const int f = c.cl.map_shared_rank(&shm, r)->found;
      if (f >= 0) last_id = f;
    }
    c.cl.sync();
  }

  // ---- the weight left, and the draw
  const double floor_w = static_cast<double>(min_p) * 17592186044416.0;  // 2^44
  // weight of id i, and whether it stays (a weight of zero may: it is then never drawn)
  auto left = [&](int i, float x, bool& stays) -> unsigned long long {
    const uint32_t k = float_order(x);
    stays = x > -INFINITY && (!cut || k > key_min || (k == key_min && c.lo + i <= last_id));
    if (!stays) return 0ull;
    const unsigned long long w = weight(x, s, shm.pw);
    stays = static_cast<double>(w) >= floor_w;
    return stays ? w : 0ull;
  };
  unsigned long long mine = 0;
  for (int i = c.wlo + lane; i < c.whi; i += 32) {
    const float x = get(i);
    bool stays;
    mine += left(i, x, stays);
    if (kept) kept[c.lo + i] = stays ? x : kCut;
  }
  mine = warp_sum_u64(mine);
  if (lane == 0) shm.warp_sum[wid] = mine;
  __syncthreads();
  if (wid == 0) {
    const unsigned long long t = warp_sum_u64(shm.warp_sum[lane]);
    if (lane == 0) shm.total = t;
  }
  c.cl.sync();
  unsigned long long total = 0, before = 0;
  for (int r = 0; r < c.ctas; ++r) {
    const unsigned long long t = c.cl.map_shared_rank(&shm, r)->total;
    if (r < c.rank) before += t;
    total += t;
  }
  for (int i = 0; i < wid; ++i) before += shm.warp_sum[i];
  const double goal = static_cast<double>(u) * static_cast<double>(total);
  // the first id whose running weight exceeds the goal; u < 1, so there is one
  if (static_cast<double>(before) <= goal && static_cast<double>(before + mine) > goal) {
    for (int i0 = c.wlo; i0 < c.whi; i0 += 32) {
      const int i = i0 + lane;
      bool stays;
      const unsigned long long w = i < c.whi ? left(i, get(i), stays) : 0ull;
      unsigned long long x = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t m = __ballot_sync(0xffffffffu, static_cast<double>(before + x) > goal);
      if (m) {
        if (lane == __ffs(m) - 1) {
          a.token[row] = c.lo + i;
          if (a.prob) a.prob[row] = static_cast<float>(static_cast<double>(w) / static_cast<double>(total));
          if (a.status) a.status[row] = 0;
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  c.cl.sync();
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st) {
  const int ctas = a.vocab > 8192 ? kMaxCtas : 1;
  const int per = (a.vocab + ctas - 1) / ctas;
  const bool held = per * 4 <= 200 * 1024;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_rows * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = held ? per * 4 : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (held) {
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = set_smem_once(sample_kernel<true>, 200 * 1024, done);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, sample_kernel<true>, a);
  }
  return cudaLaunchKernelEx(&cfg, sample_kernel<false>, a);
}

}  // namespace df2
