// Attention of new tokens over a paged cache: the kernel for few query rows per KV head
// (decoding, verify blocks, small trees), whose bound is the cache's bytes.
//
// out = softmax(scale q K^T) V in one pass over the keys: per row a running maximum m and
// sum l in base 2, o <- o 2^(m - m') + sum 2^(z - m') v.
//
//  * A KV head's query rows (new tokens x group) share every key read: one or two row
//    tiles of 16 (the MMA's M) per unit.
//  * The launch's key tiles are dealt to the CTAs in contiguous equal runs (paged.h), so
//    ragged batches and single long requests fill the machine alike; a unit cut between
//    CTAs leaves fp32 partials, joined in CTA order (whoever joins them, the same bits).
//  * Tiles of 64 keys (128 of 8 bits) come by 16-byte cp.async, zero-filled past the visible range; the
//    page table is read one tile ahead of the copies, so its latency is off the path, and
//    a tile may cross any number of pages.
//  * Four warps: one row tile x four key groups of the tile, or two x two, each with its own
//    running state, joined through shared memory when the unit (or the run) ends.  (Both row
//    tiles in one warp, so that a key's codes are converted once, was slower: 32 rows of 16
//    requests over 8192 int8 positions 142 us against 109, the second tile's registers
//    costing the third buffer.)
//  * 16-bit caches feed mma.sync through ldmatrix.  8-bit codes are exact in fp16, so both
//    products run on fp16 codes: the keys' scale multiplies the score, and the values'
//    scale the weight, relative to the largest that the row sees (so the fp16 weight
//    cannot overflow and loses at most 2^-25 of the largest); the queries are rounded to fp16
//    after an exact power-of-two shift of their row.  A lane loads the codes as 16-byte
//    pieces and the contraction order (keys) and the output columns (values) are permuted
//    to match, so no code passes through shared memory twice.
//
// Measured: 64 single tokens of 32 query heads over 8 KV heads' e4m3 caches, ragged to 16384 positions (1.34 GB): 256 to
// 268 us by the GPU, 5.0 to 5.2 TB/s, 74 to 77% of a copy's rate; DRAM moves 15% more than that, the scales' 32-byte
// sectors being read once per head.
// 16 blocks of 8 over int8 caches ragged to 8192 (0.21 GB): 85 us, bound by the latency of 8 warps an SM
// (3 us per tile of 128 keys; 0.44 instructions a scheduler and clock).  16 requests over 8192 bf16 positions (0.54 GB):
// of 4 tokens 105 us, 5.1 TB/s, of 8 (both row tiles) 108, 5.0 TB/s.
#include "common.cuh"
#include "paged_mma.cuh"
#include "paged_sched.cuh"

namespace df2 {
namespace {

constexpr int kThreads = 128;
constexpr float kGrow = 8.f;  // a row's reference follows its maximum when that has grown by more than 2^8

DF2_DEV void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
DF2_DEV void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
DF2_DEV uint4 lds16(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}
DF2_DEV uint2 lds8(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr) : "memory");
  return r;
}
template <bool BF>
DF2_DEV void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF) mma_bf16(d, a[0], a[1], a[2], a[3], b0, b1);
  else mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
}
// FMT: cache format; QBF: queries and output in bf16 (else fp16); MT: 16-row tiles per unit.
template <int D, int FMT, int MT>
struct Geo {
  static constexpr bool kQuant = FMT == kKvInt8 || FMT == kKvE4m3;
  static constexpr int kBN = kQuant ? 128 : 64;        // keys of a tile (32 KB of keys and values at D = 128)
  static constexpr int kRowBytes = D * (kQuant ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;       // 16-byte pieces of a key
  static constexpr int kSide = kBN * kRowBytes;        // keys (or values) of a tile
  static constexpr int kScales = kQuant ? 2 * kBN * 4 : 0;
  static constexpr int kStage = 2 * kSide + kScales;
  static constexpr int kStages = 3;
  static constexpr int kRows = 16 * MT;
  static constexpr int kKG = 4 / MT;                   // key groups (a warp: one row tile, one group)
  static constexpr int kWK = kBN / kKG;                // keys of a warp
  static constexpr int kNT = D / 8;                    // output column tiles
  static constexpr int kMergeCols = kNT / 4;           // column tiles joined at a time
  static constexpr int kMerge = (kKG - 1) * MT * kMergeCols * 4 * 32 * 4;
  static constexpr int kStat = 4 * 32 * 16;
  static constexpr int kOff = (kStages + 1) * kBN * 8 + (kStages + 1) * 16 + 64;
  static constexpr int kFixed = kStages * kStage + kMerge + kStat + kOff;
};

// One warp joins row lr of a cut unit (KV head h, row tile qt of the request with rows b0 .. b0 + n - 1 new tokens): the
// partials of CTAs c0 .. c1 (c0's in its slot `first`) are added in CTA order, eight at a time (their loads
// together: what this costs is latency).
template <int D, bool QBF>
DF2_DEV void join_row(const PagedAttnArgs& a, int h, int qt, int c0, int c1, int slot0, int b0, int n, int lr) {
  const int R = a.s.rows, lane = threadIdx.x & 31, row = qt * R + lr;
  if (row >= n * a.s.group) return;
  const long long first = 2ll * c0 + slot0, stride = static_cast<long long>(R) * (D + 2);
  constexpr int V = D / 32;  // channels per lane
      float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = 0.f;
      for (int c = c0; c <= c1; c += 8) {
        float2 st[8];
        float x[8][V];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          st[i] = make_float2(-INFINITY, 0.f);
          if (c + i <= c1) {
            const float* p = a.part + (c + i == c0 ? first : 2ll * (c + i)) * stride;
            st[i] = __ldcg(reinterpret_cast<const float2*>(p + R * D + 2 * lr));
            if constexpr (V == 4) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(p + lr * D + 4 * lane));
              x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
            } else {
              const float2 v = __ldcg(reinterpret_cast<const float2*>(p + lr * D + 2 * lane));
              x[i][0] = v.x, x[i][1] = v.y;
            }
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) x[i][e] = 0.f;
          }
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, st[i].x);
        const float ref = top == -INFINITY ? 0.f : top, f0 = ex2(m - ref);
        m = top;
        l *= f0;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] *= f0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = ex2(st[i].x - ref);
          l += st[i].y * f;
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] += x[i][e] * f;
        }
      }
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      const int i = row / a.s.group, head = h * a.s.group + row % a.s.group;
      char* po = a.out.p + ((b0 + i) * a.out.token_stride + head * a.out.head_stride + V * lane) * 2;
      if constexpr (V == 4)
        *reinterpret_cast<uint2*>(po) = make_uint2(pack2<QBF>(o[0] * inv, o[1] * inv), pack2<QBF>(o[2] * inv, o[3] * inv));
      else
        *reinterpret_cast<uint32_t*>(po) = pack2<QBF>(o[0] * inv, o[1] * inv);
      if (a.lse && lane == 0)
        a.lse[static_cast<long long>(b0 + i) * (a.c.n_kv * a.s.group) + head] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945f;
}

template <int D, int FMT, int MT, bool QBF>
__global__ void __launch_bounds__(kThreads, 2) paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  using G = Geo<D, FMT, MT>;
  constexpr bool kQuant = G::kQuant;
  constexpr bool kBF = kQuant ? false : QBF;  // operand type of both products
  constexpr int S = G::kStages, KG = G::kKG, WK = G::kWK, NT = G::kNT, kBN = G::kBN;
  constexpr int kSteps = D / 16;
  extern __shared__ __align__(128) char sm[];
  const uint32_t ring = smem_addr(sm);
  float* const merge = reinterpret_cast<float*>(sm + S * G::kStage);
  float4* const stat = reinterpret_cast<float4*>(sm + S * G::kStage + G::kMerge);
  long long* const offs = reinterpret_cast<long long*>(sm + S * G::kStage + G::kMerge + G::kStat);  // [S + 1][kBN]
  int* const badp = reinterpret_cast<int*>(offs + (S + 1) * kBN);                                    // [S + 1][4]
  long long* const tmp = reinterpret_cast<long long*>(badp + (S + 1) * 4);
  unsigned* const last_sh = reinterpret_cast<unsigned*>(tmp + 7);
  long long* const pre = tmp + 8;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, q = lane & 3;
  const int rg = wid % MT, kg = wid / MT;

  pdl_trigger();
  const long long T = paged_scan<kThreads>(a, pre, tmp);
  // (no empty runs: a cut unit's CTAs are then consecutive)
  const long long C = T < gridDim.x ? T : gridDim.x, c = blockIdx.x;
  if (MT > 1 && tid == 0) a.desc[8 * c] = -1;
  if (c >= C) return;
  const long long t_begin = paged_run_begin(c, C, T), t_end = paged_run_begin(c + 1, C, T);

  // ---- the page rows of a tile: one key for each of the first kBN threads.  The page table is read (fetch)
  // one tile before its entries become offsets (resolve), so that its latency lies under a tile's work.
  PagedCursor oc;
  oc.start(a, pre, t_begin, t_end);
  PagedCursor cc = oc;  // the tile that is worked on
  long long my_off = kNoRow, my_soff = 0;
  int my_bad = 0;
  int pg = 0, pg_row = 0, pg_h = 0, pg_r = 0;
  bool pg_in = false;
  auto fetch = [&]() {  // tile oc; advances oc
    pg_in = false;
    if (!oc.valid()) return;
    if (tid < kBN) {
      const int key = (oc.u.t0 + oc.i) * kBN + tid;
      pg_in = key >= oc.u.lo && key < oc.u.hi;
      if (pg_in) {
        const int pi = key / a.c.page_size;
        pg_row = key - pi * a.c.page_size;
        pg_h = oc.h;
        pg_r = oc.r;
        pg = __ldg(a.c.table + oc.r * a.c.table_stride + pi);
      }
    }
    oc.next(a);
  };
  auto resolve = [&]() {
    my_off = kNoRow;
    my_bad = 0;
    if (pg_in && !paged_row(a.c, pg, pg_row, pg_h, &my_off, &my_soff)) {
      my_bad = 1;
      if (a.rq.status) a.rq.status[pg_r] = 1;  // DFLASH2_E_INVAL
    }
  };
  auto put = [&](int slot) {  // into a slot of the offsets' ring
    if (tid < kBN) {
      offs[slot * kBN + tid] = my_off;
      const int any = __any_sync(0xffffffffu, my_bad);
      if (lane == 0) badp[4 * slot + wid] = any;
    }
  };
  long long soff_next = 0;
  bool sval_next = false;
  // A thread copies piece ch of keys r0, r0 + kStep, ...: the swizzles' key bits are its own constants.
  constexpr int kStep = kThreads / G::kChunks, kCount = kBN / kStep;
  static_assert(kStep % 8 == 0, "a thread's keys share their place in the swizzle");
  const int ch = tid % G::kChunks, r0 = tid / G::kChunks;
  const uint32_t put_k = r0 * G::kRowBytes + 16 * (kQuant ? (D == 128 ? ch ^ ((r0 & 1) << 2) : ch) : ch ^ (r0 & 7));
  const uint32_t put_v = G::kSide + r0 * G::kRowBytes +
                         16 * (kQuant ? (D == 128 ? ch ^ (r0 & 6) : ch ^ ((r0 >> 1) & 3)) : ch ^ (r0 & 7));
  auto issue = [&](int stage, int slot) {  // the copies of a tile whose offsets are in `slot`
    const uint32_t dst = ring + stage * G::kStage;
    const long long* o = offs + slot * kBN + r0;
    long long off[kCount];
#pragma unroll
    for (int i = 0; i < kCount; ++i) off[i] = o[i * kStep];
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const bool in = off[i] != kNoRow;
      const int bytes = in ? 16 : 0;
      const long long byte = (in ? off[i] * (kQuant ? 1 : 2) : 0) + ch * 16;
      cp_async16(dst + put_k + i * (kStep * G::kRowBytes), a.c.k + byte, bytes);
      cp_async16(dst + put_v + i * (kStep * G::kRowBytes), a.c.v + byte, bytes);
    }
    if constexpr (kQuant) {
      if (tid < kBN) {
        cp_async4(dst + 2 * G::kSide + tid * 4, a.c.k_scale + soff_next, sval_next ? 4 : 0);
        cp_async4(dst + 2 * G::kSide + kBN * 4 + tid * 4, a.c.v_scale + soff_next, sval_next ? 4 : 0);
      }
    }
  };

  const int n_tiles = static_cast<int>(t_end - t_begin);
  // prologue: tiles 0 .. S - 2 in flight, the offsets of tile S - 1 looked up
#pragma unroll
  for (int j = 0; j < S - 1; ++j) {
    fetch();
    resolve();
    put(j);
    soff_next = my_soff;
    sval_next = my_off != kNoRow;
    __syncthreads();
    if (j < n_tiles) issue(j, j);
    cp_commit();
  }
  fetch();
  resolve();
  put(S - 1);
  soff_next = my_soff;
  sval_next = my_off != kNoRow;
  fetch();  // tile S

  uint32_t qf[kSteps][4];
  float o[NT][4];
  float m0 = 0, m1 = 0, l0 = 0, l1 = 0, sc0 = 0, sc1 = 0, vref0 = 0, vref1 = 0;
  uint32_t nan0 = 0, nan1 = 0;  // channels of the two rows with a code of NaN that they see
  int hi0 = 0, hi1 = 0, lo0 = 0, lo1 = 0, base = 0;       // visible keys of this thread's two rows
  int hi_min = 0, lo_max = 0;                             // keys in [lo_max, hi_min) are visible to every row
  bool mixed_rows = false;
  unsigned long long w0 = 0, w1 = 0;
  bool fresh = true;
  int st_now = 0, st_next = S - 1;       // stages of tiles j and j + S - 1
  int sl_now = 0, sl_next = S - 1;       // offset slots of the same (ring of S + 1); tile j + S takes the one after

  for (int j = 0; j < n_tiles; ++j) {
    if (fresh) {
      fresh = false;
      const int rows = cc.n * a.s.group;
      const int ra = cc.qt * G::kRows + rg * 16 + g, rb = ra + 8;
      base = cc.len - cc.n;
      const int ia = ra / a.s.group, ib = rb / a.s.group;
      const bool va = ra < rows, vb = rb < rows;
      hi0 = va ? (a.s.causal == 1 ? min(cc.len, base + ia + 1) : cc.len) : 0;
      hi1 = vb ? (a.s.causal == 1 ? min(cc.len, base + ib + 1) : cc.len) : 0;
      lo0 = a.s.window > 0 ? base + ia - a.s.window + 1 : 0;
      lo1 = a.s.window > 0 ? base + ib - a.s.window + 1 : 0;
      if (a.s.causal == 2) {
        w0 = va ? __ldg(a.tree + cc.b0 + ia) : 0ull;
        w1 = vb ? __ldg(a.tree + cc.b0 + ib) : 0ull;
      }
      const int i_first = cc.qt * G::kRows / a.s.group;
      const int i_last = (min((cc.qt + 1) * G::kRows, rows) - 1) / a.s.group;
      hi_min = a.s.causal == 1 ? min(cc.len, base + i_first + 1) : (a.s.causal == 2 ? min(cc.len, base) : cc.len);
      lo_max = a.s.window > 0 ? base + i_last - a.s.window + 1 : 0;
      mixed_rows = i_last > i_first || a.s.causal == 2;
      const char* pa = a.q.p + ((cc.b0 + ia) * a.q.token_stride + (cc.h * a.s.group + ra % a.s.group) * a.q.head_stride) * 2;
      const char* pb = a.q.p + ((cc.b0 + ib) * a.q.token_stride + (cc.h * a.s.group + rb % a.s.group) * a.q.head_stride) * 2;
      if constexpr (!kQuant) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          qf[s][0] = va ? *reinterpret_cast<const uint32_t*>(pa + (16 * s + 2 * q) * 2) : 0u;
          qf[s][1] = vb ? *reinterpret_cast<const uint32_t*>(pb + (16 * s + 2 * q) * 2) : 0u;
          qf[s][2] = va ? *reinterpret_cast<const uint32_t*>(pa + (16 * s + 2 * q + 8) * 2) : 0u;
          qf[s][3] = vb ? *reinterpret_cast<const uint32_t*>(pb + (16 * s + 2 * q + 8) * 2) : 0u;
        }
        sc0 = sc1 = a.scale_log2;
      } else {
        // step 4 h + w, slots 2 q, 2 q + 1 and 2 q + 8, 2 q + 9 hold channels 16 (q + 4 h) + 4 w + 0 .. 3
        float xa = 0.f, xb = 0.f;
#pragma unroll
        for (int hh = 0; hh < kSteps / 4; ++hh) {
#pragma unroll
          for (int w = 0; w < 4; w += 2) {
            const int d = 16 * (q + 4 * hh) + 4 * w;
            const uint4 ua = va ? *reinterpret_cast<const uint4*>(pa + d * 2) : make_uint4(0, 0, 0, 0);
            const uint4 ub = vb ? *reinterpret_cast<const uint4*>(pb + d * 2) : make_uint4(0, 0, 0, 0);
            qf[4 * hh + w][0] = ua.x, qf[4 * hh + w][2] = ua.y, qf[4 * hh + w + 1][0] = ua.z, qf[4 * hh + w + 1][2] = ua.w;
            qf[4 * hh + w][1] = ub.x, qf[4 * hh + w][3] = ub.y, qf[4 * hh + w + 1][1] = ub.z, qf[4 * hh + w + 1][3] = ub.w;
          }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<QBF>(qf[s][e]);
            float& x = (e & 1) ? xb : xa;
            x = fmaxf(x, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
#pragma unroll
        for (int of = 1; of <= 2; of <<= 1) {
          xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, of));
          xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, of));
        }
        // (to fp16, the codes' exact type: exact from 2^-14 of the row's largest on, off by at most 2^-25 of that below)
        const float fa = pow2_shift(xa), fb = pow2_shift(xb);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<QBF>(qf[s][e]);
            const float m = (e & 1) ? fb : fa;
            qf[s][e] = pack2<false>(f.x * m, f.y * m);
          }
        sc0 = a.scale_log2 / fa;
        sc1 = a.scale_log2 / fb;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
      vref0 = vref1 = 0x1p-126f;
      nan0 = nan1 = 0;
    }

    cp_wait<S - 2>();
    __syncthreads();  // tile j has landed; tile j - 1's buffer and the offsets of tile j + S - 1 are free / written
    if (j + S - 1 < n_tiles) issue(st_next, sl_next);
    cp_commit();
    resolve();  // tile j + S
    fetch();    // tile j + S + 1

    const uint32_t ks = ring + st_now * G::kStage, vs = ks + G::kSide;
    const float* ksc = reinterpret_cast<const float*>(sm + st_now * G::kStage + 2 * G::kSide);
    const float* vsc = ksc + kBN;
    const int key0 = (cc.u.t0 + cc.i) * kBN;
    const int* bad = badp + 4 * sl_now;
    const bool any_bad = (bad[0] | bad[1] | (kBN > 64 ? bad[2] | bad[3] : 0)) != 0;
    const bool masked = key0 < lo_max || key0 + kBN > hi_min || any_bad;
    const int kw = kg * WK;  // keys kw .. kw + WK - 1 of the tile

    // ---- scores
    float z[WK / 8][4];
#pragma unroll
    for (int t = 0; t < WK / 8; ++t) z[t][0] = z[t][1] = z[t][2] = z[t][3] = 0.f;
    if constexpr (!kQuant) {
#pragma unroll
      for (int t = 0; t < WK / 8; t += 2) {
        const int row = kw + 8 * t + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          uint32_t b[4];
          ldsm4(b, ks + row * G::kRowBytes + (((2 * s + ((lane >> 3) & 1)) ^ (row & 7)) << 4));
          mma16<kBF>(z[t], qf[s], b[0], b[1]);
          mma16<kBF>(z[t + 1], qf[s], b[2], b[3]);
        }
      }
    } else {
#pragma unroll
      for (int t = 0; t < WK / 8; ++t) {
        const uint32_t row = ks + (kw + 8 * t + g) * G::kRowBytes;
#pragma unroll
        for (int hh = 0; hh < kSteps / 4; ++hh) {
          const int c16 = q + 4 * hh;
          const uint4 w = lds16(row + ((D == 128 ? c16 ^ ((g & 1) << 2) : c16) << 4));
          mma16<false>(z[t], qf[4 * hh + 0], codes2<FMT, 0>(w.x), codes2<FMT, 1>(w.x));
          mma16<false>(z[t], qf[4 * hh + 1], codes2<FMT, 0>(w.y), codes2<FMT, 1>(w.y));
          mma16<false>(z[t], qf[4 * hh + 2], codes2<FMT, 0>(w.z), codes2<FMT, 1>(w.z));
          mma16<false>(z[t], qf[4 * hh + 3], codes2<FMT, 0>(w.w), codes2<FMT, 1>(w.w));
        }
      }
    }
    // ---- scale, mask, running reference
#pragma unroll
    for (int t = 0; t < WK / 8; ++t) {
      float2 f = make_float2(1.f, 1.f);
      if constexpr (kQuant) f = *reinterpret_cast<const float2*>(ksc + kw + 8 * t + 2 * q);
      z[t][0] *= sc0 * f.x, z[t][1] *= sc0 * f.y;
      z[t][2] *= sc1 * f.x, z[t][3] *= sc1 * f.y;
    }
    auto sees = [&](int key, bool& v0, bool& v1) {  // this thread's two rows
      v0 = key >= lo0 && key < hi0, v1 = key >= lo1 && key < hi1;
      if (a.s.causal == 2 && key >= base) {
        v0 = v0 && ((w0 >> ((key - base) & 63)) & 1ull);
        v1 = v1 && ((w1 >> ((key - base) & 63)) & 1ull);
      }
    };
    if (masked) {
#pragma unroll
      for (int t = 0; t < WK / 8; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int kk = kw + 8 * t + 2 * q + e;
          bool v0, v1;
          sees(key0 + kk, v0, v1);
          if (any_bad && offs[sl_now * kBN + kk] == kNoRow) v0 = v1 = false;
          z[t][e] = v0 ? z[t][e] : -INFINITY;
          z[t][2 + e] = v1 ? z[t][2 + e] : -INFINITY;
        }
    }
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int t = 0; t < WK / 8; ++t) {
      x0 = fmaxf(x0, fmaxf(z[t][0], z[t][1]));
      x1 = fmaxf(x1, fmaxf(z[t][2], z[t][3]));
    }
#pragma unroll
    for (int of = 1; of <= 2; of <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, of));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, of));
    }
    // O and the sum are rescaled only when a maximum has grown by more than 2^8 (weights stay below 2^8)
    float f0 = 1.f, f1 = 1.f;
    if (x0 > m0 + kGrow) {
      f0 = ex2(m0 - x0);
      m0 = x0;
    }
    if (x1 > m1 + kGrow) {
      f1 = ex2(m1 - x1);
      m1 = x1;
    }
    l0 *= f0;
    l1 *= f1;
    // a row that has seen nothing keeps weights of zero: 2^(-inf - 0)
    const float ref0 = m0 == -INFINITY ? 0.f : m0, ref1 = m1 == -INFINITY ? 0.f : m1;
    if constexpr (kQuant) {
      // the row's reference follows the largest finite scale of this warp's keys that the row sees; where rows differ each
      // looks at its own keys (one that it does not see costs it nothing)
      float v0 = 0.f, v1 = 0.f;
      if (masked && mixed_rows) {
#pragma unroll
        for (int t = 0; t < WK / 8; ++t) {
          const float2 f = *reinterpret_cast<const float2*>(vsc + kw + 8 * t + 2 * q);
          const float fx = f.x < INFINITY ? f.x : 0.f, fy = f.y < INFINITY ? f.y : 0.f;
          if (z[t][0] != -INFINITY) v0 = fmaxf(v0, fx);
          if (z[t][1] != -INFINITY) v0 = fmaxf(v0, fy);
          if (z[t][2] != -INFINITY) v1 = fmaxf(v1, fx);
          if (z[t][3] != -INFINITY) v1 = fmaxf(v1, fy);
        }
#pragma unroll
        for (int of = 1; of <= 2; of <<= 1) {
          v0 = fmaxf(v0, __shfl_xor_sync(0xffffffffu, v0, of));
          v1 = fmaxf(v1, __shfl_xor_sync(0xffffffffu, v1, of));
        }
      } else {
#pragma unroll
        for (int i = 0; i < WK; i += 32) {
          const float y = vsc[kw + i + lane];
          v0 = y < INFINITY ? fmaxf(v0, y) : v0;
        }
        v0 = v1 = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v0)));  // (ordered as the floats from 0 are)
      }
      if (v0 > kMostFactor * vref0) {
        const float v = scale_reference(v0);
        f0 *= vref0 * reciprocal(v);
        vref0 = v;
      }
      if (v1 > kMostFactor * vref1) {
        const float v = scale_reference(v1);
        f1 *= vref1 * reciprocal(v);
        vref1 = v;
      }
    }
    if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        o[t][0] *= f0;
        o[t][1] *= f0;
        o[t][2] *= f1;
        o[t][3] *= f1;
      }
    }
    // ---- weights and the values' product.  The sum takes the weights in fp32; the product rounds them once to its
    // operands' type, which has to be the values' (bf16, or fp16 where the codes are), off by 2^-8 or 2^-11 of a weight at most.
    // In two pieces they would cost the product twice.  Against 64 bits (relative error of the outputs, bf16 caches; that of
    // rounding the output alone 0.0017): 0.0019 for a single token, 0.0023 for trees; 8 bits: 0.0017.
    const float vinv0 = reciprocal(vref0), vinv1 = reciprocal(vref1);
#pragma unroll
    for (int t = 0; t < WK / 8; ++t) {
      const bool h0 = z[t][0] == -INFINITY, h1 = z[t][1] == -INFINITY, h2 = z[t][2] == -INFINITY, h3 = z[t][3] == -INFINITY;
      const float p0 = ex2(z[t][0] - ref0), p1 = ex2(z[t][1] - ref0), p2 = ex2(z[t][2] - ref1), p3 = ex2(z[t][3] - ref1);
      l0 += p0 + p1;
      l1 += p2 + p3;
      z[t][0] = p0, z[t][1] = p1, z[t][2] = p2, z[t][3] = p3;
      if constexpr (kQuant) {
        const float2 f = *reinterpret_cast<const float2*>(vsc + kw + 8 * t + 2 * q);
        z[t][0] *= f.x * vinv0, z[t][1] *= f.y * vinv0;
        z[t][2] *= f.x * vinv1, z[t][3] *= f.y * vinv1;
        if (masked) {  // (a masked position's scale may be anything)
          if (h0) z[t][0] = 0.f;
          if (h1) z[t][1] = 0.f;
          if (h2) z[t][2] = 0.f;
          if (h3) z[t][3] = 0.f;
        }
      }
    }
    // Values may be infinities or NaN (8 bits: codes of NaN) at positions that only some rows see: there the
    // product takes zeros in their place, and each is added to the rows that see it, however small their weight (8 bits:
    // noted for them)
    bool poison = false;
    if constexpr (!kQuant || FMT == kKvE4m3) {
      if (masked && mixed_rows) {
        bool bad_v = false;
        constexpr uint32_t ex = kBF ? 0x7F80u : 0x7C00u;
        for (int i = lane; i < WK * G::kChunks; i += 32) {
          const uint4 w = lds16(vs + kw * G::kRowBytes + i * 16);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int u = 0; u < 4; ++u)
            bad_v |= kQuant ? nan_codes(ww[u]) != 0 : (ww[u] & ex) == ex || ((ww[u] >> 16) & ex) == ex;
        }
        poison = kQuant ? __syncthreads_or(bad_v) != 0 : __any_sync(0xffffffffu, bad_v) != 0;
      }
    }
    if (poison) {
      if constexpr (!kQuant) {
#pragma unroll
        for (int t = 0; t < WK / 8; ++t) {
          for (int qq = 0; qq < 4; ++qq) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = kw + 8 * t + 2 * qq + e;
              bool v0, v1;
              sees(key0 + row, v0, v1);
#pragma unroll
              for (int d = 0; d < NT; ++d) {
                uint32_t w;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(vs + row * G::kRowBytes + ((d ^ (row & 7)) << 4) + 4 * q) : "memory");
                const float2 v = unpack2<kBF>(w);
                if (!isfinite(v.x)) {
                  if (v0) o[d][0] += v.x;
                  if (v1) o[d][2] += v.x;
                }
                if (!isfinite(v.y)) {
                  if (v0) o[d][1] += v.y;
                  if (v1) o[d][3] += v.y;
                }
              }
            }
          }
        }
      } else {
        // this thread's channels, D / 8 from (D / 8) (2 q + e) on, in the rows that see them; then zeros in the codes' place
#pragma unroll 1
        for (int kk = kw; kk < kw + WK; ++kk) {
          bool v0, v1;
          sees(key0 + kk, v0, v1);
#pragma unroll 1
          for (int c = 0; c < NT / 2; ++c) {  // words
            const int cw = q * (NT / 2) + c;
            uint32_t x;
            asm volatile("ld.shared.u32 %0, [%1];"
                         : "=r"(x)
                         : "r"(vs + kk * G::kRowBytes + (((cw >> 2) ^ (D == 128 ? kk & 6 : (kk >> 1) & 3)) << 4) + ((cw & 3) << 2))
                         : "memory");
            x = nan_codes(x) & 0x08040201u;
            const uint32_t bits = ((x | x >> 8) | (x | x >> 8) >> 16) & 15u;
            if (v0) nan0 |= bits << (4 * c);
            if (v1) nan1 |= bits << (4 * c);
          }
        }
        __syncthreads();
        for (int i = tid; i < kBN * G::kChunks; i += kThreads) {
          const uint4 w = lds16(vs + i * 16);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(vs + i * 16), "r"(w.x & ~nan_codes(w.x)),
                       "r"(w.y & ~nan_codes(w.y)), "r"(w.z & ~nan_codes(w.z)), "r"(w.w & ~nan_codes(w.w))
                       : "memory");
        }
        __syncthreads();
      }
    }
    {
#pragma unroll
      for (int kk = 0; kk < WK / 16; ++kk) {
        const uint32_t pf[4] = {pack2<kBF>(z[2 * kk][0], z[2 * kk][1]), pack2<kBF>(z[2 * kk][2], z[2 * kk][3]),
                                pack2<kBF>(z[2 * kk + 1][0], z[2 * kk + 1][1]),
                                pack2<kBF>(z[2 * kk + 1][2], z[2 * kk + 1][3])};
        if constexpr (!kQuant) {
          const int row = kw + 16 * kk + (lane & 15);
#pragma unroll
          for (int t = 0; t < NT; t += 2) {
            uint32_t b[4];
            ldsm4_t(b, vs + row * G::kRowBytes + (((t + (lane >> 4)) ^ (row & 7)) << 4));
            if (poison) {
#pragma unroll
              for (int i = 0; i < 4; ++i) b[i] = finite2<kBF>(b[i]);
            }
            mma16<kBF>(o[t], pf, b[0], b[1]);
            mma16<kBF>(o[t + 1], pf, b[2], b[3]);
          }
        } else {
          const int row = kw + 16 * kk + 2 * q;
          uint32_t r[4][NT / 4];  // codes of channels (D / 8) g .. of keys row, row + 1, row + 8, row + 9
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = row + (i & 1) + ((i >> 1) << 3);
            if constexpr (D == 128) {
              const uint4 w = lds16(vs + rr * G::kRowBytes + ((g ^ (rr & 6)) << 4));
              r[i][0] = w.x, r[i][1] = w.y, r[i][2] = w.z, r[i][3] = w.w;
            } else {
              const uint2 w = lds8(vs + rr * G::kRowBytes + (((g >> 1) ^ ((rr >> 1) & 3)) << 4) + (g & 1) * 8);
              r[i][0] = w.x, r[i][1] = w.y;
            }
          }
#pragma unroll
          for (int w = 0; w < NT / 4; ++w) {
            const uint32_t ab = __byte_perm(r[0][w], r[1][w], 0x5140), ab2 = __byte_perm(r[0][w], r[1][w], 0x7362);
            const uint32_t cd = __byte_perm(r[2][w], r[3][w], 0x5140), cd2 = __byte_perm(r[2][w], r[3][w], 0x7362);
            mma16<false>(o[4 * w + 0], pf, codes2<FMT, 0>(ab), codes2<FMT, 0>(cd));
            mma16<false>(o[4 * w + 1], pf, codes2<FMT, 1>(ab), codes2<FMT, 1>(cd));
            mma16<false>(o[4 * w + 2], pf, codes2<FMT, 0>(ab2), codes2<FMT, 0>(cd2));
            mma16<false>(o[4 * w + 3], pf, codes2<FMT, 1>(ab2), codes2<FMT, 1>(cd2));
          }
        }
      }
    }

    sl_next = sl_next == S ? 0 : sl_next + 1;
    put(sl_next);
    soff_next = my_soff;
    sval_next = my_off != kNoRow;
    sl_now = sl_now == S ? 0 : sl_now + 1;
    st_now = st_now == S - 1 ? 0 : st_now + 1;
    st_next = st_next == S - 1 ? 0 : st_next + 1;

    // ---- end of the unit or of the run: join the key groups, write
    const bool last = j == n_tiles - 1;
    if (cc.unit_ends() || last) {
      if constexpr (kQuant) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          o[t][0] *= vref0, o[t][1] *= vref0;
          o[t][2] *= vref1, o[t][3] *= vref1;
        }
        if (FMT == kKvE4m3 && (nan0 | nan1)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if ((nan0 >> (e * NT + t)) & 1u) o[t][e] = NAN;
              if ((nan1 >> (e * NT + t)) & 1u) o[t][2 + e] = NAN;
            }
        }
      }
#pragma unroll
      for (int of = 1; of <= 2; of <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, of);
        l1 += __shfl_xor_sync(0xffffffffu, l1, of);
      }
      {
        stat[wid * 32 + lane] = make_float4(m0, m1, l0, l1);
        __syncthreads();
        float y0 = m0, y1 = m1;
#pragma unroll
        for (int i = 0; i < KG; ++i) {
          const float4 st = stat[(i * MT + rg) * 32 + lane];
          y0 = fmaxf(y0, st.x);
          y1 = fmaxf(y1, st.y);
        }
        const float b0 = y0 == -INFINITY ? 0.f : y0, b1 = y1 == -INFINITY ? 0.f : y1;
        const float e0 = ex2(m0 - b0), e1 = ex2(m1 - b1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          o[t][0] *= e0;
          o[t][1] *= e0;
          o[t][2] *= e1;
          o[t][3] *= e1;
        }
        l0 = l1 = 0.f;
#pragma unroll
        for (int i = 0; i < KG; ++i) {
          const float4 st = stat[(i * MT + rg) * 32 + lane];
          l0 += st.z * ex2(st.x - b0);
          l1 += st.w * ex2(st.y - b1);
        }
        m0 = y0;
        m1 = y1;
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          constexpr int MC = G::kMergeCols;
          if (part) __syncthreads();
          if (kg > 0) {
#pragma unroll
            for (int t = 0; t < MC; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) merge[((((kg - 1) * MT + rg) * MC + t) * 4 + e) * 32 + lane] = o[part * MC + t][e];
          }
          __syncthreads();
          if (kg == 0) {
#pragma unroll
            for (int i = 0; i < KG - 1; ++i)
#pragma unroll
              for (int t = 0; t < MC; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[part * MC + t][e] += merge[(((i * MT + rg) * MC + t) * 4 + e) * 32 + lane];
          }
        }
        // the buffers are next written after the next tile's barrier
      }
      if (kg == 0) {
        const int rows = cc.n * a.s.group;
        const bool whole = cc.unit_t >= t_begin && cc.unit_ends();
        const long long slot = 2 * c + (cc.unit_t <= t_begin ? 0 : 1);
        if (MT > 1 && !whole && tid == 0 && cc.unit_t >= t_begin) {  // the cut unit begins here: tell the combine
          const long long tl = cc.unit_t + cc.u.nt;
          long long cb = (tl * C - 1) / T;  // the CTA of the unit's last tile
          int* dd = a.desc + 8 * c;
          dd[1] = cc.h;
          dd[2] = cc.qt;
          dd[3] = static_cast<int>(cb) * 2 + (cc.unit_t == t_begin ? 0 : 1);
          dd[4] = cc.b0;
          dd[5] = cc.n;
          dd[0] = cc.r;
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int lr = rg * 16 + g + 8 * hf, row = cc.qt * G::kRows + lr;
          if (row >= rows) continue;
          const float l = hf ? l1 : l0, m = hf ? m1 : m0;
          if (whole) {
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (a NaN sum stays NaN)
            const int i = row / a.s.group, head = cc.h * a.s.group + row % a.s.group;
            char* po = a.out.p + ((cc.b0 + i) * a.out.token_stride + head * a.out.head_stride) * 2;
            if constexpr (!kQuant) {
#pragma unroll
              for (int t = 0; t < NT; ++t)
                *reinterpret_cast<uint32_t*>(po + (8 * t + 2 * q) * 2) =
                    pack2<QBF>(o[t][2 * hf] * inv, o[t][2 * hf + 1] * inv);
            } else {
              // this thread's columns: (D / 8) (2 q + e) + t
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int t = 0; t < NT; t += 8)
                  *reinterpret_cast<uint4*>(po + (NT * (2 * q + e) + t) * 2) = make_uint4(
                      pack2<QBF>(o[t][2 * hf + e] * inv, o[t + 1][2 * hf + e] * inv),
                      pack2<QBF>(o[t + 2][2 * hf + e] * inv, o[t + 3][2 * hf + e] * inv),
                      pack2<QBF>(o[t + 4][2 * hf + e] * inv, o[t + 5][2 * hf + e] * inv),
                      pack2<QBF>(o[t + 6][2 * hf + e] * inv, o[t + 7][2 * hf + e] * inv));
            }
            if (a.lse && q == 0)
              a.lse[static_cast<long long>(cc.b0 + i) * (a.c.n_kv * a.s.group) + head] =
                  l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945f;
          } else {
            float* pp = a.part + slot * (G::kRows * (D + 2)) + lr * D;
            if constexpr (!kQuant) {
#pragma unroll
              for (int t = 0; t < NT; ++t)
                *reinterpret_cast<float2*>(pp + 8 * t + 2 * q) = make_float2(o[t][2 * hf], o[t][2 * hf + 1]);
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int t = 0; t < NT; t += 4)
                  *reinterpret_cast<float4*>(pp + NT * (2 * q + e) + t) =
                      make_float4(o[t][2 * hf + e], o[t + 1][2 * hf + e], o[t + 2][2 * hf + e], o[t + 3][2 * hf + e]);
            }
            if (q == 0)
              *reinterpret_cast<float2*>(a.part + slot * (G::kRows * (D + 2)) + G::kRows * D + 2 * lr) = make_float2(m, l);
          }
        }
      }
      if constexpr (MT == 1) {
        // one row tile: the CTA that brings a cut unit's last partial joins them (up to four rows a warp), which saves a
        // launch; the counter wraps to zero by itself
        if (cc.unit_t < t_begin || !cc.unit_ends()) {
          const int c0 = cc.unit_t >= t_begin ? static_cast<int>(c) : static_cast<int>(((cc.unit_t + 1) * C - 1) / T);
          const int c1 = static_cast<int>(((cc.unit_t + cc.u.nt) * C - 1) / T);
          __threadfence();  // this thread's partials before the count
          __syncthreads();
          if (tid == 0) *last_sh = atomicInc(a.count + c0, c1 - c0) == static_cast<unsigned>(c1 - c0);
          __syncthreads();
          if (*last_sh) {
            __threadfence();
            const int slot0 = paged_run_begin(c0, C, T) == cc.unit_t ? 0 : 1;
            for (int lr = wid; lr < G::kRows; lr += kThreads / 32)
              join_row<D, QBF>(a, cc.h, cc.qt, c0, c1, slot0, cc.b0, cc.n, lr);
          }
        }
      }
      fresh = true;
    }
    cc.next(a);
  }
}

// Flags every request with a tile in CTA c's run (a wait of that CTA gave up).
DF2_DEV void flag_run(const PagedAttnArgs& a, long long c) {
  if (!a.rq.status) return;
  auto tiles = [&](int r) {
    int b0, n, len;
    return paged_request(a.rq, r, b0, n, len) ? a.c.n_kv * paged_head_tiles(a.s, n, len) : 0ll;
  };
  long long T = 0, first = 0;
  for (int r = 0; r < a.rq.n_req; ++r) T += tiles(r);
  const long long C = T < gridDim.x ? T : gridDim.x;
  for (int r = 0; r < a.rq.n_req; ++r) {
    const long long next = first + tiles(r);
    if (paged_in_run(first, next, paged_run_begin(c, C, T), paged_run_begin(c + 1, C, T))) a.rq.status[r] = 3;  // DFLASH2_E_CUDA
    first = next;
  }
}

// Joins the partials of the units cut between CTAs, where the attention leaves that to a launch of its own.  WAITS: of the
// kernel for many rows, whose waits may give up.
template <int D, bool QBF, bool WAITS>
__global__ void __launch_bounds__(128) paged_combine_kernel(const __grid_constant__ PagedAttnArgs a) {
  pdl_wait();  // (launched while the attention still runs)
  const int4 d0 = *reinterpret_cast<const int4*>(a.desc + 8 * blockIdx.x);
  const int4 d1 = *reinterpret_cast<const int4*>(a.desc + 8 * blockIdx.x + 4);
  if (WAITS && d1.z != 0 && blockIdx.y == 0 && threadIdx.x == 0) flag_run(a, blockIdx.x);
  if (d0.x < 0) return;
  for (int lr = blockIdx.y * 4 + (threadIdx.x >> 5); lr < a.s.rows; lr += 4 * gridDim.y)
    join_row<D, QBF>(a, d0.y, d0.z, blockIdx.x, d0.w >> 1, d0.w & 1, d1.x, d1.y, lr);
}

template <int D, int FMT, int MT, bool QBF>
cudaError_t launch_rows(PagedAttnArgs& a, int num_sms, cudaStream_t st) {
  using G = Geo<D, FMT, MT>;
  a.s.bn = G::kBN;
  static std::atomic<unsigned long long> done{0};
  const int smem = G::kFixed + (a.rq.n_req + 1 + 8) * 8;
  cudaError_t e = set_smem_once(paged_attn_kernel<D, FMT, MT, QBF>, G::kFixed + (1024 + 16) * 8, done);
  if (e != cudaSuccess) return e;
  const int per_sm = kPagedMaxCtasPerSm;
  // no more CTAs than tiles there can be
  const long long rt = (static_cast<long long>(a.rq.max_new) * a.s.group + G::kRows - 1) / G::kRows;
  const long long most = static_cast<long long>(a.rq.n_req) * a.c.n_kv * rt * ((a.rq.max_len + G::kBN - 1) / G::kBN + 1);
  a.ctas = static_cast<int>(most < static_cast<long long>(num_sms) * per_sm ? most : num_sms * per_sm);
  paged_attn_kernel<D, FMT, MT, QBF><<<a.ctas, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int D, int FMT, bool QBF>
cudaError_t launch_fmt(PagedAttnArgs& a, int num_sms, cudaStream_t st) {
  a.s.rows = paged_rows(a.rq.max_new, a.s.group);
  return a.s.rows == 16 ? launch_rows<D, FMT, 1, QBF>(a, num_sms, st) : launch_rows<D, FMT, 2, QBF>(a, num_sms, st);
}

template <int D>
cudaError_t launch_dim(PagedAttnArgs& a, int fmt, int qtype, int num_sms, cudaStream_t st) {
  const bool bf = qtype == kTBf16;
  switch (fmt) {
    case kKvBf16: return launch_fmt<D, kKvBf16, true>(a, num_sms, st);
    case kKvF16: return launch_fmt<D, kKvF16, false>(a, num_sms, st);
    case kKvInt8: return bf ? launch_fmt<D, kKvInt8, true>(a, num_sms, st) : launch_fmt<D, kKvInt8, false>(a, num_sms, st);
    default: return bf ? launch_fmt<D, kKvE4m3, true>(a, num_sms, st) : launch_fmt<D, kKvE4m3, false>(a, num_sms, st);
  }
}

}  // namespace

cudaError_t launch_paged_attention(PagedAttnArgs& a, int head_dim, int fmt, int qtype, int num_sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.rq.max_new) * a.s.group;
  cudaError_t e;
  if (rows > kChunkMinRows) e = launch_paged_chunk(a, head_dim, fmt, qtype, num_sms, st);
  else e = head_dim == 64 ? launch_dim<64>(a, fmt, qtype, num_sms, st) : launch_dim<128>(a, fmt, qtype, num_sms, st);
  if (e != cudaSuccess || a.s.rows == 16) return e;  // (one row tile: joined by the kernel itself)
  // a row per warp for units of 32 rows (four in turn took 2 to 3 us more), four for those of 256
  const dim3 grid(a.ctas, a.s.rows == 32 ? 8 : a.s.rows / 16);
  auto combine = [&](auto kernel, auto kernel_waits) {
    return launch_ex(a.s.rows == 32 ? kernel : kernel_waits, grid, dim3(128), 0, st, true, a);
  };
  if (head_dim == 64)
    return qtype == kTBf16 ? combine(paged_combine_kernel<64, true, false>, paged_combine_kernel<64, true, true>)
                           : combine(paged_combine_kernel<64, false, false>, paged_combine_kernel<64, false, true>);
  return qtype == kTBf16 ? combine(paged_combine_kernel<128, true, false>, paged_combine_kernel<128, true, true>)
                         : combine(paged_combine_kernel<128, false, false>, paged_combine_kernel<128, false, true>);
}

}  // namespace df2
