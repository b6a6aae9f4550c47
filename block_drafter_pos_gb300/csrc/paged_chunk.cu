// Attention of new tokens over a paged cache: the kernel for many query rows per KV head
// (prompt chunks, large trees), on the fifth-generation tensor cores.
//
// A unit is 256 rows of one KV head (two tiles of 128: the MMA's M) against its visible keys in
// tiles of 128; units and runs are dealt as in the kernel for few rows (paged.h), so a chunk's
// causal triangle, ragged prompts and few heads all load the machine evenly.
//
//  * S = Q K^T and O += P V are tcgen05.mma with fp32 accumulators in tensor memory: S of the
//    two row tiles in columns 0 .. 255, O in 256 .. 511.  P (16 bit) overwrites the first half of
//    its S and is read by the MMA from there; Q, K, V lie in shared memory under the
//    128-byte swizzle, V as the MN-major operand, so it needs no transposition.
//  * Warps 0 - 3 and 4 - 7 own a row tile each, one row per thread: running maximum and sum in
//    registers, no shuffles.  O is rescaled only when a row's maximum has grown by more than
//    2^8 (weights then stay below 2^8, within range of either 16-bit type, and the fp32 sums lose
//    nothing), which after a unit's first tiles is rare; the tile's own warps do it.
//  * While one tile's weights are being computed the tensor core works on the other's
//    products: one thread of warp 12 issues O0, S0', O1, S1', ...
//  * Warps 8 - 11 bring the keys and values: cp.async of 16-byte pieces through the page table
//    (any page size; its rows are looked up one tile ahead), or, for 8-bit caches, cp.async of the
//    codes into a staging area from which the same thread writes them as exact fp16 values.  The
//    keys' scale multiplies the score and the values' scale the weight, relative to a
//    reference that is raised when a scale exceeds 128 of it (row by row where rows see different keys).
//  * Every wait is bounded; one that gives up marks the CTA and ends it once its own copies and
//    products are done.  The kernel that joins partials flags the run's requests; rows whose partials never came are NaN.
//
// Measured: 4096 new tokens of 32 query heads over 32768 bf16 positions of 8 KV heads of 128 (2.06 TFLOP): 1.68 to
// 1.75 ms, 1.2 PFLOP/s, 69 to 72% of the sustained cuBLAS rate, tensor pipe 52% active.  A 128-key tile takes about
// 3900 clocks where its products take 2048: a row tile's softmax (1700), the products of its weights and next scores
// (1024) and the hand-offs between them follow one another, and two row tiles cover only part of each other.
// Five chunks of 1501 tokens of 24 heads of 64 over e4m3 caches with a window of 2048: 245 us, bound by the softmax's
// instructions (a scale and a factor for every key besides the exponential; tensor pipe 18% active), 19 of them the join.
// Under the launch's 128 registers 16-bit caches spill 12 bytes a thread and 8-bit ones 92 to 128 (read back: 72, and 284 to
// 320).
#include "common.cuh"
#include "paged_mma.cuh"
#include "paged_sched.cuh"
#include "pipeline.cuh"

namespace df2 {
namespace {

using pipe::lds128;
using pipe::mbar_arrive;
using pipe::mbar_init_count;
using pipe::mbar_wait;
using pipe::smem_u32;

constexpr int kThreads = 512;
constexpr int kLoaders = 128;
constexpr int kSoftRegs = 200, kOtherRegs = 56;  // 256 threads each: the 512 x 128 of the launch
constexpr int kBN = kChunkBn;      // keys per tile
constexpr int kM = 128;            // rows per tile
constexpr float kGrow = 8.f;       // log2 of the largest weight
// References of the values' scales in a wide tile (below).  A row's is at least 2^-112: weights over it, and sums of 128 of
// them, stay finite, and what smaller values lose in fp16 weights is below 2^-126.  The tile's is at most 2^20, so that the
// weights of rows with references from 2^-92 to 2^120 are summed over it.
constexpr float kLeastRef = 0x1p-112f, kMostRef = 0x1p20f;

template <int D, int FMT>
struct ChunkGeo {
  static constexpr bool kQuant = FMT == kKvInt8 || FMT == kKvE4m3;
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * 128 * 128;        // a 16-bit operand tile
  static constexpr int kSlots = kQuant ? 3 : 4;
  static constexpr int kOffRing = 2 * kTile;
  static constexpr int kOffStage = kOffRing + kSlots * kTile;
  static constexpr int kStage = kQuant ? 128 * D : 0;      // codes of a tile
  static constexpr int kBufs = kQuant ? (D == 64 ? 4 : 2) : 0;
  // operands copied ahead of the one that is announced (16 bits: two ahead was slower, 1.79 ms against 1.66 for a
  // 4096-token chunk over 32768 keys: a full ring then holds back what has landed)
  static constexpr int kLag = kQuant ? kBufs - 1 : 1;
  static constexpr int kOffInfo = kOffStage + kBufs * kStage;
  // tile information, a ring of 8: key scales, value factors, bad-page bits, value reference
  static constexpr int kRing = 8;
  static constexpr int kInfo = 128 * 4 * 2 + 16 + 16;
  static constexpr int kOffOffs = kOffInfo + kRing * kInfo;    // element offsets of a tile's keys, two tiles
  static constexpr int kOffPre = kOffOffs + 2 * 128 * 8;   // tiles before each request
  static constexpr int kFixed = kOffPre + 1024;            // + alignment
};

// Shared-memory matrix descriptors under the 128-byte swizzle: the low words hold the address and the
// leading offset, the high word is the same for all (8-row groups 1024 bytes apart, this architecture's
// version, the swizzle).  K-major tiles (queries, keys): rows of 64 channels; the leading offset is not used.
// MN-major (values): rows of 64 channels, 8 keys per atom; the next 64 channels are the leading offset on.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
DF2_DEV uint32_t desc_k(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
DF2_DEV uint32_t desc_mn(uint32_t saddr) { return (saddr >> 4) | ((16384u >> 4) << 16); }
__host__ __device__ constexpr uint32_t instr(bool bf, int n, bool b_mn) {
  const uint32_t ab = bf ? 1u : 0u;
  return (1u << 4) | (ab << 7) | (ab << 10) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kM >> 4) << 24);
}
// The products are issued by one lane (`go`) of a warp that stays converged, so that the descriptors live in
// uniform registers.
DF2_DEV void mma_ss(uint32_t go, uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %6, 0;\n mov.b64 x, {%1, %5};\n"
      " mov.b64 y, {%2, %5};\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHi), "r"(go)
      : "memory");
}
DF2_DEV void mma_ts(uint32_t go, uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %6, 0;\n mov.b64 y, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHi), "r"(go)
      : "memory");
}
DF2_DEV void mma_commit(uint32_t go, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(go)
      : "memory");
}
// mbar_wait of a whole warp, its loop out of the compiler's sight (1 if the phase completed within the limit).
DF2_DEV uint32_t mbar_wait_warp(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n .reg .u32 i;\n mov.u32 i, 0;\n mov.u32 %0, 1;\n"
      "AGAIN:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra DONE;\n add.u32 i, i, 1;\n"
      " setp.lt.u32 p, i, %3;\n @p bra AGAIN;\n mov.u32 %0, 0;\nDONE:\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity), "n"(static_cast<int>(pipe::kSpinLimit))
      : "memory");
  return done;
}
DF2_DEV void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
DF2_DEV void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
DF2_DEV void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

DF2_DEV void tm_ld32(uint32_t t, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]),
        "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]),
        "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]),
        "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(t));
}
DF2_DEV void tm_ld16(uint32_t t, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]),
        "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(t));
}
DF2_DEV void tm_st16(uint32_t t, const float* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]),
      "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
      : "memory");
}
template <typename V>
DF2_DEV void tm_st32(uint32_t t, const V* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
DF2_DEV void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
DF2_DEV void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
DF2_DEV void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
DF2_DEV void loaders_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// What a unit's rows see, as ranges: keys in [lo_max, hi_min) are visible to every row.
struct UnitMask {
  int base, hi_min, lo_max;
  bool mixed;  // rows differ (or a tree decides key by key)
  DF2_DEV void set(const PagedShape& s, const PagedCursor& c) {
    base = c.len - c.n;
    const int rows = c.n * s.group, i0 = c.qt * s.rows / s.group;
    const int i1 = (min((c.qt + 1) * s.rows, rows) - 1) / s.group;
    hi_min = s.causal == 1 ? min(c.len, base + i0 + 1) : (s.causal == 2 ? min(c.len, base) : c.len);
    lo_max = s.window > 0 ? base + i1 - s.window + 1 : 0;
    mixed = i1 > i0 || s.causal == 2;
  }
  DF2_DEV bool masked(int key0) const { return key0 < lo_max || key0 + kBN > hi_min; }
};

// 64 columns as bits: those below n, and a word whose bit 0 is column n.
DF2_DEV unsigned long long columns_below(int n) { return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull); }
DF2_DEV unsigned long long columns_shifted(unsigned long long w, int n) {
  return n >= 64 || n <= -64 ? 0ull : (n >= 0 ? w << n : w >> -n);
}

template <int D, int FMT, bool QBF>
__global__ void __launch_bounds__(kThreads, 1) paged_chunk_kernel(const __grid_constant__ PagedAttnArgs a) {
  using G = ChunkGeo<D, FMT>;
  constexpr bool kQuant = G::kQuant;
  constexpr bool kBF = kQuant ? false : QBF;
  constexpr int NS = G::kSlots;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[NS * 2 + G::kRing + 11];
  __shared__ uint32_t tmem_sh;
  // By unit: the number (from 1) of the last unit in the slot some of whose values are not finite.  Numbers only
  // grow, so a row tile that is still at an older unit finds at worst a newer one's, and looks in vain.
  __shared__ int poison_sh[G::kRing];
  __shared__ long long tmp[kThreads / 32 + 1];
  __shared__ float vmax_sh[2][4], vmin_sh[2][4];
  __shared__ int flag_sh[2][4];
  static_assert(256 * (kSoftRegs + kOtherRegs) == kThreads * 128, "the register split");
  const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* const sgen = smem_raw + (sbase - smem_u32(smem_raw));
  const uint32_t full = smem_u32(bars), empty = full + 8 * NS, info = empty + 8 * NS, s_full = info + 8 * G::kRing,
                 p_full = s_full + 16, q_full = p_full + 32, o_done = q_full + 16, all_done = o_done + 16;
  long long* const pre = reinterpret_cast<long long*>(sgen + G::kOffPre);
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init_count(full + 8 * i, kLoaders);
      mbar_init_count(empty + 8 * i, 1);
    }
    for (int i = 0; i < G::kRing; ++i) {
      mbar_init_count(info + 8 * i, kLoaders);
      poison_sh[i] = 0;
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init_count(s_full + 8 * t, 1);
      mbar_init_count(p_full + 16 * t, 4);
      mbar_init_count(p_full + 16 * t + 8, 4);
      mbar_init_count(q_full + 8 * t, 4);
      mbar_init_count(o_done + 8 * t, 1);
    }
    mbar_init_count(all_done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_trigger();
  const long long T = paged_scan<kThreads>(a, pre, tmp);
  const long long C = T < gridDim.x ? T : gridDim.x, c = blockIdx.x;
  if (tid == 0) a.desc[8 * c] = -1, a.desc[8 * c + 6] = 0;
  if (c >= C) return;
  const long long t_begin = paged_run_begin(c, C, T), t_end = paged_run_begin(c + 1, C, T);
  // Partials that never come (a wait that gives up) leave NaN in the rows they are joined into.
  for (int i = tid; i < 2 * kChunkRows; i += kThreads) {
    float* const p = a.part + (2 * c + i / kChunkRows) * (kChunkRows * (D + 2)) + kChunkRows * D;
    reinterpret_cast<float2*>(p)[i % kChunkRows] = make_float2(NAN, NAN);
  }
  if (wid == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_sh)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_sh;
  bool ok = true;

  if (wid < 8) {
    // ---------------------------------------------------------------- weights of row tile t
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int t = wid >> 2, lrow = tid & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((wid & 3) * 32) << 16);
    const uint32_t s_col = lane_base + 128 * t, o_col = lane_base + 256 + 128 * t;
    PagedCursor cc;
    cc.start(a, pre, t_begin, t_end);
    int n = 0, gtile = 0, gunit = 0;  // this row tile's key tiles so far; the run's key tiles and units
    float m = -INFINITY, l = 0.f, sc = 0.f, vref = 0.f;
    int lo = 0, hi = 0;
    unsigned long long word = 0;
    UnitMask um;
    bool active = false;
    // This row's query of the cursor's unit into shared memory (the row tile's scores so far are complete, so
    // its former queries have been read), and what the row sees.
    auto enter = [&](const PagedCursor& u) {
      const int rows = u.n * a.s.group - u.qt * a.s.rows;  // of the unit (may exceed it)
      active = t == 0 || rows > kM;
      um.set(a.s, u);
      if (!active) return;
      const int row = u.qt * a.s.rows + t * kM + lrow;
      const bool valid = t * kM + lrow < rows;
      const int i = row / a.s.group, head = u.h * a.s.group + row % a.s.group;
      hi = valid ? (a.s.causal == 1 ? min(u.len, um.base + i + 1) : u.len) : 0;
      lo = a.s.window > 0 ? max(um.base + i - a.s.window + 1, 0) : 0;
      if (a.s.causal == 2) word = valid ? __ldg(a.tree + u.b0 + i) : 0ull;
      const uint4* p = reinterpret_cast<const uint4*>(a.q.p + ((u.b0 + i) * a.q.token_stride + head * a.q.head_stride) * 2);
      uint4 w[D / 8];
#pragma unroll
      for (int x = 0; x < D / 8; ++x) w[x] = valid ? __ldg(p + x) : make_uint4(0, 0, 0, 0);
      // The score's factor stays above 0, so that a masked score stays -infinity: the query takes the scale's sign, and a
      // scale of 0 itself.
      const float sign = a.scale_log2 == 0.f ? 0.f : (a.scale_log2 < 0.f ? -1.f : 1.f);
      sc = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
      if constexpr (kQuant) {
        float x = 0.f;
#pragma unroll
        for (int y = 0; y < D / 8; ++y) {
          const uint32_t ww[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<QBF>(ww[e]);
            x = fmaxf(x, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        // (to fp16, the codes' exact type: exact from 2^-14 of the row's largest on, off by at most 2^-25 of that below)
        const float f = pow2_shift(x);
        sc = fmaxf(sc / f, 0x1p-149f);
#pragma unroll
        for (int y = 0; y < D / 8; ++y) {
          uint32_t ww[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = unpack2<QBF>(ww[e]);
            ww[e] = pack2<false>(v.x * (f * sign), v.y * (f * sign));
          }
          w[y] = make_uint4(ww[0], ww[1], ww[2], ww[3]);
        }
      } else if (sign == 0.f) {
#pragma unroll
        for (int y = 0; y < D / 8; ++y)
          w[y] = make_uint4(times_zero2<kBF>(w[y].x), times_zero2<kBF>(w[y].y), times_zero2<kBF>(w[y].z), times_zero2<kBF>(w[y].w));
      } else if (sign < 0.f) {
#pragma unroll
        for (int y = 0; y < D / 8; ++y)
          w[y] = make_uint4(w[y].x ^ 0x80008000u, w[y].y ^ 0x80008000u, w[y].z ^ 0x80008000u, w[y].w ^ 0x80008000u);
      }
      const uint32_t q = sbase + t * G::kTile + lrow * 128;
#pragma unroll
      for (int x = 0; x < D / 8; ++x) sts128(q + (x >> 3) * 16384 + (((x & 7) ^ (lrow & 7)) << 4), w[x]);
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + 8 * t);
    };
    // The columns of the key tile at key0 that the row sees, one bit each.
    auto visible = [&](int key0, int flags, const uint32_t* badw, unsigned long long& v0, unsigned long long& v1) {
      v0 = columns_below(hi - key0) & ~columns_below(lo - key0);
      v1 = columns_below(hi - key0 - 64) & ~columns_below(lo - key0 - 64);
      if (a.s.causal == 2) {
        const int d = um.base - key0;  // the column of the tree's first token
        v0 &= columns_below(d) | columns_shifted(word, d);
        v1 &= columns_below(d - 64) | columns_shifted(word, d - 64);
      }
      if (flags & 1) {
        v0 &= ~(static_cast<unsigned long long>(badw[1]) << 32 | badw[0]);
        v1 &= ~(static_cast<unsigned long long>(badw[3]) << 32 | badw[2]);
      }
    };
    enter(cc);
    while (cc.valid() && ok) {
      const int piece = cc.piece();
      for (int j = 0; active && j < piece; ++j) {
        // ---- scores of one key tile
        const int key0 = (cc.u.t0 + cc.i + j) * kBN;
        const int ring = (gtile + j) % G::kRing;
        const float* ks = reinterpret_cast<const float*>(sgen + G::kOffInfo + ring * G::kInfo);
        const float* vf = ks + 128;
        const uint32_t* badw = reinterpret_cast<const uint32_t*>(vf + 128);
        // (the scores' products follow the tile's information, whose barrier is then in this use's phase)
        ok = mbar_wait(s_full + 8 * t, static_cast<uint32_t>(n & 1)) &&
             mbar_wait(info + 8 * ring, static_cast<uint32_t>(((gtile + j) / G::kRing) & 1));
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        fence_after();
        float s[128];
#pragma unroll
        for (int x = 0; x < 4; ++x) tm_ld32(s_col + 32 * x, s + 32 * x);
        // the tile's information: whether some page is bad, the values' reference
        const int2 fl = *reinterpret_cast<const int2*>(badw + 4);
        tm_wait_ld();
        if constexpr (kQuant) {
          float4 w[4], v[4];  // 16 keys' scales, and the next 16
#pragma unroll
          for (int y = 0; y < 4; ++y) w[y] = *reinterpret_cast<const float4*>(ks + 4 * y);
#pragma unroll
          for (int x = 0; x < 128; x += 16) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (x + 16 < 128) v[y] = *reinterpret_cast<const float4*>(ks + x + 16 + 4 * y);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int e = x + 4 * y;
              const float2 y0 = mul2(make_float2(s[e], s[e + 1]), make_float2(w[y].x, w[y].y));
              const float2 y1 = mul2(make_float2(s[e + 2], s[e + 3]), make_float2(w[y].z, w[y].w));
              s[e] = y0.x, s[e + 1] = y0.y, s[e + 2] = y1.x, s[e + 3] = y1.y;
              w[y] = v[y];
            }
          }
        }
        const bool masked = um.masked(key0) || (fl.x & 1);
        if (masked) {
          unsigned long long v0, v1;
          visible(key0, fl.x, badw, v0, v1);
          const uint32_t vw[4] = {static_cast<uint32_t>(v0), static_cast<uint32_t>(v0 >> 32), static_cast<uint32_t>(v1),
                                  static_cast<uint32_t>(v1 >> 32)};
#pragma unroll
          for (int x = 0; x < 128; ++x) s[x] = (vw[x >> 5] >> (x & 31)) & 1u ? s[x] : -INFINITY;
        }
        float x0 = s[0], x1 = s[1], x2 = s[2], x3 = s[3];
#pragma unroll
        for (int x = 4; x < 124; x += 8) {
          x0 = fmaxf(fmaxf(x0, s[x]), s[x + 4]);
          x1 = fmaxf(fmaxf(x1, s[x + 1]), s[x + 5]);
          x2 = fmaxf(fmaxf(x2, s[x + 2]), s[x + 6]);
          x3 = fmaxf(fmaxf(x3, s[x + 3]), s[x + 7]);
        }
        x0 = fmaxf(fmaxf(x0, s[124]), x2);
        x1 = fmaxf(fmaxf(x1, s[125]), x3);
        const float mx = fmaxf(fmaxf(fmaxf(x0, s[126]), s[127]), x1) * sc;
        float f = 1.f;  // O's factor
        const bool fresh = j == 0 || m == -INFINITY;  // (nothing seen so far)
        if (j == 0) {
          m = mx;
        } else if (mx > m + kGrow) {
          f = ex2(m - mx);
          m = mx;
          l *= f;
        }
        // The values' scales are relative to the tile's reference, which is the unit's, and so is O: unless rows of the
        // tile differ and its scales are too far apart for one.  Then (a wide tile) each row takes a reference of its
        // own, the tile's by a power of two near a 16th of the largest scale that it sees, so that one it does not
        // see costs it nothing; and it goes back to the unit's in the next tile, if that is not so far below that the
        // weights there are nothing.
        // The tile's reference over the row's: its exponent, which the weights take, and its reciprocal.
        float rowe = 0.f, rowi = 1.f;
        if constexpr (kQuant) {
          const float tref = __int_as_float(fl.y);
          if (fresh) vref = tref;
          if (vref != tref || (fl.x & 2)) {
            float v = tref, r = 1.f;
            if (vref > 0x1p64f * tref) {  // (no weight is above fp16's least)
              v = vref;
              r = 0x1p-60f;
            }
            if ((fl.x & 2) && !(vref > 0x1p108f * tref)) {
              unsigned long long v0, v1;
              visible(key0, fl.x, badw, v0, v1);
              v = 0.f;
#pragma unroll 1
              for (int x = 0; x < 128; x += 4) {
                const float4 w = *reinterpret_cast<const float4*>(vf + x);
                const uint32_t b = static_cast<uint32_t>((x < 64 ? v0 : v1) >> (x & 63));
                v = fmaxf(v, fmaxf(fmaxf(b & 1 ? w.x : 0.f, b & 2 ? w.y : 0.f), fmaxf(b & 4 ? w.z : 0.f, b & 8 ? w.w : 0.f)));
              }
              const float per = reciprocal(tref);
              float rel = pow2_at(fmaxf(v * 0.0625f, kLeastRef * fmaxf(1.f, per)));
              const float now = pow2_at(vref * per);
              if (!fresh && v <= kMostFactor * now) rel = now;
              v = tref * rel;
              // (at less than 2^-60 no weight is above fp16's least, unless the factors are large)
              r = fmaxf(pow2_inverse(rel), tref < kMostRef ? 0x1p-60f : 0x1p-126f);
            }
            if (!fresh) f *= vref * reciprocal(v);
            vref = v;
            rowe = pow2_exponent(r);
            rowi = pow2_inverse(r);
          }
        }
        if (__any_sync(0xffffffffu, f != 1.f)) {
          ok = mbar_wait(o_done + 8 * t, static_cast<uint32_t>((n - 1) & 1));
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          fence_after();
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            float o[16];
            tm_ld16(o_col + 16 * x, o);
            tm_wait_ld();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] *= f;
            tm_st16(o_col + 16 * x, o);
          }
        }
        // ---- weights (a row that has seen nothing: 2^(-infinity)), announced by halves.  Rounded once, after their sum
        // has taken them in fp32, to the product's operand type, which has to be the values': errors against 64 bits 0.0023
        // with bf16 where the output's own rounding is 0.0017, 0.00029 with fp16 where that is 0.00021.
        const float mr0 = m == -INFINITY ? 0.f : -m, mr = kQuant ? mr0 + rowe : mr0;
        float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
        const float2 sc2 = make_float2(sc, sc), mr2 = make_float2(mr, mr);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t p[32];
          float4 w[4], v[4];  // 16 keys' value factors, and the next 16
          if constexpr (kQuant) {
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = *reinterpret_cast<const float4*>(vf + 64 * x + 4 * y);
          }
#pragma unroll
          for (int y0 = 0; y0 < 32; y0 += 8) {
            if constexpr (kQuant) {
#pragma unroll
              for (int y = 0; y < 4; ++y)
                if (y0 + 8 < 32) v[y] = *reinterpret_cast<const float4*>(vf + 64 * x + 2 * y0 + 16 + 4 * y);
            }
#pragma unroll
            for (int y = y0; y < y0 + 8; y += 2) {
              const int e = 64 * x + 2 * y;
              float2 a0 = fma2(make_float2(s[e], s[e + 1]), sc2, mr2), a1 = fma2(make_float2(s[e + 2], s[e + 3]), sc2, mr2);
              a0 = make_float2(ex2(a0.x), ex2(a0.y));
              a1 = make_float2(ex2(a1.x), ex2(a1.y));
              acc0 = add2(acc0, a0);
              acc1 = add2(acc1, a1);
              if constexpr (kQuant) {
                const float4 f4 = w[(y - y0) / 2];
                const float2 b0 = mul2(a0, make_float2(f4.x, f4.y)), b1 = mul2(a1, make_float2(f4.z, f4.w));
                p[y] = pack2<kBF>(b0.x, b0.y);
                p[y + 1] = pack2<kBF>(b1.x, b1.y);
                w[(y - y0) / 2] = v[(y - y0) / 2];
              } else {
                p[y] = pack2<kBF>(a0.x, a0.y);
                p[y + 1] = pack2<kBF>(a1.x, a1.y);
              }
            }
          }
          tm_st32(s_col + 32 * x, p);
          tm_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 8 * (2 * t + x));
        }
        acc0 = add2(acc0, acc1);
        l += (acc0.x + acc0.y) * (kQuant ? rowi : 1.f);
        ++n;
      }
      if (!ok) break;
      // ---- the end of the unit (or of the run): the next unit's queries first, then this one's outputs
      PagedCursor nc = cc;
      nc.skip(a, piece);
      {
        const int old_lo = lo, old_hi = hi;
        const unsigned long long old_word = word;
        const UnitMask old_um = um;
        const bool was_active = active;
        if (nc.valid()) enter(nc);
        if (was_active) {
          const int rows = cc.n * a.s.group - cc.qt * a.s.rows;
          const int i_last = cc.i + piece - 1;
          const bool whole = cc.unit_t >= t_begin && i_last == cc.u.nt - 1;
          const long long slot = 2 * c + (cc.unit_t <= t_begin ? 0 : 1);
          if (!whole && t == 0 && lrow == 0 && cc.unit_t >= t_begin) {  // the cut unit begins here: tell the combine
            const long long cb = ((cc.unit_t + cc.u.nt) * C - 1) / T;
            int* dd = a.desc + 8 * c;
            dd[1] = cc.h;
            dd[2] = cc.qt;
            dd[3] = static_cast<int>(cb) * 2 + (cc.unit_t == t_begin ? 0 : 1);
            dd[4] = cc.b0;
            dd[5] = cc.n;
            dd[0] = cc.r;
          }
          ok = mbar_wait(o_done + 8 * t, static_cast<uint32_t>((n - 1) & 1));
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          fence_after();
          const int lr = t * kM + lrow, row = cc.qt * a.s.rows + lr;
          const bool valid = lr < rows;
          const int i = row / a.s.group, head = cc.h * a.s.group + row % a.s.group;
          const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (a NaN sum stays NaN)
          const float out_f = kQuant ? (whole ? inv * vref : vref) : (whole ? inv : 1.f);
          char* const po = a.out.p + ((cc.b0 + i) * a.out.token_stride + head * a.out.head_stride) * 2;
          float* const pp = a.part + slot * (a.s.rows * (D + 2)) + lr * D;
          const bool poison = *static_cast<volatile int*>(&poison_sh[gunit % G::kRing]) > gunit;
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            float o[32];
            __syncwarp();
            tm_ld32(o_col + 32 * x, o);
            tm_wait_ld();
            if (poison && valid) {
              // values that are not finite: the product had zeros there (16 bits, and 8-bit codes of NaN: in tiles where
              // rows differ; 8 bits: where the scale is not finite)
              const int first_i = cc.unit_t >= t_begin ? 0 : static_cast<int>(t_begin - cc.unit_t);
              for (int ti = first_i; ti <= i_last; ++ti) {
                const int k0 = (cc.u.t0 + ti) * kBN;
                if (!kQuant && !old_um.masked(k0)) continue;
                for (int key = max(k0, old_lo); key < min(k0 + kBN, old_hi); ++key) {
                  if (a.s.causal == 2 && key >= old_um.base && !((old_word >> (key - old_um.base)) & 1ull)) continue;
                  const int page = __ldg(a.c.table + cc.r * a.c.table_stride + key / a.c.page_size);
                  long long off, so;
                  if (!paged_row(a.c, page, key % a.c.page_size, cc.h, &off, &so)) continue;
                  if constexpr (kQuant) {
                    const float vs = __ldg(a.c.v_scale + so);
                    const bool fine = fabsf(vs) < INFINITY;
                    if (fine && !(FMT == kKvE4m3 && old_um.mixed && old_um.masked(k0))) continue;
                    const uint32_t* v = reinterpret_cast<const uint32_t*>(a.c.v + off + 32 * x);
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                      uint32_t w = __ldg(v + y);
                      if (fine) w &= nan_codes(w);  // (of the other codes 0)
                      const float2 v0 = unpack2<false>(codes2<FMT, 0>(w)), v1 = unpack2<false>(codes2<FMT, 1>(w));
                      o[4 * y] += v0.x * vs, o[4 * y + 1] += v0.y * vs, o[4 * y + 2] += v1.x * vs, o[4 * y + 3] += v1.y * vs;
                    }
                  } else {
                    const uint32_t* v = reinterpret_cast<const uint32_t*>(a.c.v + (off + 32 * x) * 2);
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                      const float2 vv = unpack2<kBF>(__ldg(v + y));
                      if (!isfinite(vv.x)) o[2 * y] += vv.x;
                      if (!isfinite(vv.y)) o[2 * y + 1] += vv.y;
                    }
                  }
                }
              }
            }
            if (valid) {
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] *= out_f;
              if (whole) {
#pragma unroll
                for (int y = 0; y < 32; y += 8)
                  *reinterpret_cast<uint4*>(po + (32 * x + y) * 2) =
                      make_uint4(pack2<QBF>(o[y], o[y + 1]), pack2<QBF>(o[y + 2], o[y + 3]), pack2<QBF>(o[y + 4], o[y + 5]),
                                 pack2<QBF>(o[y + 6], o[y + 7]));
              } else {
#pragma unroll
                for (int y = 0; y < 32; y += 4)
                  *reinterpret_cast<float4*>(pp + 32 * x + y) = make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
              }
            }
          }
          if (valid) {
            if (whole) {
              if (a.lse)
                a.lse[static_cast<long long>(cc.b0 + i) * (a.c.n_kv * a.s.group) + head] =
                    l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945f;
            } else {
              *reinterpret_cast<float2*>(a.part + slot * (a.s.rows * (D + 2)) + a.s.rows * D + 2 * lr) = make_float2(m, l);
            }
          }
          __syncwarp();
          fence_before();  // O has been read before this tile's next weights are announced
        }
        m = -INFINITY;
        l = 0.f;
      }
      ++gunit;
      gtile += piece;
      cc = nc;
    }
    if (!ok && lane == 0) a.desc[8 * c + 6] = 1;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (wid == 12) {
      // -------------------------------------------------------------- products
      const uint32_t go = lane == 0 ? 1u : 0u;
      constexpr uint32_t id_s = instr(kBF, kBN, false), id_o = instr(kBF, D, true);
      PagedCursor cs;  // the unit whose scores come next
      cs.start(a, pre, t_begin, t_end);
      const int total = static_cast<int>(t_end - t_begin);
      int sn = 0, units = 0, left = cs.piece(), piece = left;  // tiles of that unit still to come
      uint32_t units1 = 0, pn0 = 0, pn1 = 0;
      uint32_t fine = 1;
      bool s_first = true;
      bool two_cur = cs.n * a.s.group - cs.qt * a.s.rows > kM, first_cur = true;  // of the tile whose weights come next
      bool two_next = two_cur;
      // scores of row tile t of key tile sn (cs's unit)
      auto scores = [&](uint32_t t, bool two) {
        const uint32_t idx = 2 * sn, slot = idx % NS;
        if (t == 0) fine &= mbar_wait_warp(full + 8 * slot, (idx / NS) & 1);
        if (s_first) fine &= mbar_wait_warp(q_full + 8 * t, (t ? units1 : units) & 1);
        fence_after();
        const uint32_t q = desc_k(sbase + t * G::kTile), kd = desc_k(sbase + G::kOffRing + slot * G::kTile);
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          mma_ss(go, tmem + 128 * t, q + (x >> 2) * 1024 + 2 * (x & 3), kd + (x >> 2) * 1024 + 2 * (x & 3), id_s, x != 0);
        mma_commit(go, s_full + 8 * t);
        if (t == 1 || !two) mma_commit(go, empty + 8 * slot);
      };
      // outputs of row tile t of key tile n
      auto outputs = [&](uint32_t t, int n, bool two, bool first) {
        const uint32_t idx = 2 * n + 1, slot = idx % NS, ph = (t ? pn1 : pn0) & 1;
        if (t == 0) fine &= mbar_wait_warp(full + 8 * slot, (idx / NS) & 1);
        fine &= mbar_wait_warp(p_full + 16 * t, ph);
        fence_after();
        const uint32_t v = desc_mn(sbase + G::kOffRing + slot * G::kTile), p = tmem + 128 * t, o = tmem + 256 + 128 * t;
#pragma unroll
        for (int x = 0; x < kBN / 32; ++x) mma_ts(go, o, p + 8 * x, v + 128 * x, id_o, x == 0 ? !first : 1);
        fine &= mbar_wait_warp(p_full + 16 * t + 8, ph);
        fence_after();
#pragma unroll
        for (int x = kBN / 32; x < kBN / 16; ++x) mma_ts(go, o, p + 8 * x, v + 128 * x, id_o, 1);
        mma_commit(go, o_done + 8 * t);
        if (t == 1 || !two) mma_commit(go, empty + 8 * slot);
        if (t) ++pn1;
        else ++pn0;
      };
      // (a failed wait ends the loop at the tile's end: the others' waits run out in turn)
      for (int n = -1; n < total; ++n) {
        const bool more = n + 1 < total;
        if (n >= 0 && more) {
          s_first = --left == 0;
          if (s_first) {
            ++units;
            if (two_next) ++units1;
            cs.skip(a, piece);
            left = piece = cs.piece();
            two_next = __any_sync(0xffffffffu, cs.n * a.s.group - cs.qt * a.s.rows > kM);
          }
          ++sn;
        }
#pragma unroll 1
        for (uint32_t t = 0; t < 2; ++t) {
          if (n >= 0 && (t == 0 || two_cur)) outputs(t, n, two_cur, first_cur);
          if (more && (t == 0 || two_next)) scores(t, two_next);
        }
        two_cur = two_next;
        first_cur = s_first;
        if (!__all_sync(0xffffffffu, fine != 0)) {
          ok = false;
          break;
        }
      }
      if (!ok && lane == 0) a.desc[8 * c + 6] = 1;
    } else if (wid < 12) {
      // -------------------------------------------------------------- keys and values
      const int lt = tid - 256;
      long long* const offs = reinterpret_cast<long long*>(sgen + G::kOffOffs);
      PagedCursor lc;
      lc.start(a, pre, t_begin, t_end);
      const int total = static_cast<int>(t_end - t_begin);
      UnitMask um;
      um.set(a.s, lc);
      long long off = kNoRow;
      float ksv = 0.f, vsv = 0.f;
      bool badv = false, piece_first = true, mixed = false, l_first = true;
      int unit = 0;
      // offset and scales of the cursor's tile for this thread's key
      auto look_up = [&]() {
        if (l_first) um.set(a.s, lc);
        const int key0 = (lc.u.t0 + lc.i) * kBN, key = key0 + lt;
        mixed = um.mixed && um.masked(key0);
        piece_first = l_first;
        off = kNoRow;
        ksv = vsv = 0.f;
        badv = false;
        if (key >= lc.u.lo && key < lc.u.hi) {
          const int pi = key / a.c.page_size;
          const int page = __ldg(a.c.table + lc.r * a.c.table_stride + pi);
          long long so;
          if (paged_row(a.c, page, key - pi * a.c.page_size, lc.h, &off, &so)) {
            if (kQuant) {
              ksv = __ldg(a.c.k_scale + so);
              vsv = __ldg(a.c.v_scale + so);
            }
          } else {
            badv = true;
            if (a.rq.status) a.rq.status[lc.r] = 1;  // DFLASH2_E_INVAL
          }
        }
        l_first = lc.unit_ends();
        lc.next(a);
      };
      float vref = 0.f, vinv = 0.f, seen_by_all = 0.f;
      look_up();
      // A thread copies piece ch of rows r0, r0 + kStep, ...: the swizzle's row bits are its own constant.
      constexpr int kPieces = D * (kQuant ? 1 : 2) / 16, kStep = kLoaders / kPieces, kCount = 128 / kStep;
      constexpr int kBatch = kCount < 8 ? kCount : 8, BUFS = G::kBufs > 0 ? G::kBufs : 1;
      const int ch = lt % kPieces, r0 = lt / kPieces;
      // where piece ch of row r0 goes (16-bit: itself; codes: the first of its two pieces of fp16)
      const int piece = kQuant ? 2 * ch : ch;
      const uint32_t put0 = (piece >> 3) * 16384 + r0 * 128 + (((piece & 7) ^ (r0 & 7)) << 4);
      const uint32_t put1 = (piece >> 3) * 16384 + r0 * 128 + ((((piece & 7) + 1) ^ (r0 & 7)) << 4);
      static_assert(kStep % 8 == 0, "a thread's rows share their place in the swizzle");
      auto landed = [&](int idx) {  // this thread's part of operand idx is in place
        fence_async();
        mbar_arrive(full + 8 * (idx % NS));
      };
      auto freed = [&](int idx) {  // the operand that had idx's slot has been read
        const int use = idx / NS;
        return use == 0 || mbar_wait(empty + 8 * (idx % NS), static_cast<uint32_t>((use + 1) & 1));
      };
      // 8-bit: this thread's codes of operand idx from the staging area to its slot; values that only some rows see without
      // codes of NaN (the rows that see them add them at the end)
      int tile = 0;                              // the tile looked up last; of it (bit 0) and those before:
      uint32_t mixed_bits = 0, first_bits = 0;   // whether rows differ in it, and whether a unit (but the first) begins
      auto convert = [&](int idx) {
        if (!freed(idx)) return false;
        if constexpr (kQuant) {
          const int age = tile - (idx >> 1);
          const bool strip = FMT == kKvE4m3 && (idx & 1) && ((mixed_bits >> age) & 1u);
          bool found = false;
          const uint32_t st = sbase + G::kOffStage + (idx % BUFS) * G::kStage + lt * 16;
          const uint32_t dst = sbase + G::kOffRing + (idx % NS) * G::kTile;
#pragma unroll
          for (int x0 = 0; x0 < kCount; x0 += 4) {
            uint4 w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] = lds128(st + (x0 + x) * (kLoaders * 16));
            if (strip) {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint4 z = make_uint4(nan_codes(w[x].x), nan_codes(w[x].y), nan_codes(w[x].z), nan_codes(w[x].w));
                found |= (z.x | z.y | z.z | z.w) != 0;
                w[x] = make_uint4(w[x].x & ~z.x, w[x].y & ~z.y, w[x].z & ~z.z, w[x].w & ~z.w);
              }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t d = dst + (x0 + x) * (kStep * 128);
              sts128(d + put0, make_uint4(codes2<FMT, 0>(w[x].x), codes2<FMT, 1>(w[x].x), codes2<FMT, 0>(w[x].y), codes2<FMT, 1>(w[x].y)));
              sts128(d + put1, make_uint4(codes2<FMT, 0>(w[x].z), codes2<FMT, 1>(w[x].z), codes2<FMT, 0>(w[x].w), codes2<FMT, 1>(w[x].w)));
            }
          }
          if (found) {
            const int u = unit - __popc(first_bits & ((1u << age) - 1u));  // the tile's unit
            poison_sh[u % G::kRing] = u + 1;
          }
        }
        landed(idx);
        return true;
      };
      int said = 0;  // operands announced
      // (after a failed wait a loader goes through the motions, so that the loaders' barrier stays whole)
      for (int j = 0; j < total; ++j) {
        // ---- the tile's information
        const int ring = j % G::kRing;
        float* ks = reinterpret_cast<float*>(sgen + G::kOffInfo + ring * G::kInfo);
        uint32_t* badw = reinterpret_cast<uint32_t*>(ks + 256);
        long long* o = offs + (j & 1) * 128;
        if (piece_first && j > 0) ++unit;
        tile = j;
        mixed_bits = mixed_bits << 1 | (mixed ? 1u : 0u);
        first_bits = first_bits << 1 | (piece_first && j > 0 ? 1u : 0u);
        // (The slot's previous tile was eight tiles ago: operands up to that of tile j - 5 have been read, or this
        // thread could not be here, so the weights of tile j - 5 are done.)
        if constexpr (kQuant) {
          const float v = warp_max(vsv < INFINITY ? vsv : 0.f);
          // (keys without a scale, outside the unit's range or on a bad page among them, count as 0 there and not at all here)
          const float w = -warp_max(vsv > 0.f && vsv < INFINITY ? -vsv : -INFINITY);
          if (lane == 0) vmax_sh[j & 1][wid - 8] = v, vmin_sh[j & 1][wid - 8] = w;
        }
        o[lt] = off;
        const uint32_t b = __ballot_sync(0xffffffffu, badv);
        if (lane == 0) {
          badw[wid - 8] = b;
          flag_sh[j & 1][wid - 8] = b ? 1 : 0;
        }
        loaders_sync();
        uint32_t flags = flag_sh[j & 1][0] | flag_sh[j & 1][1] | flag_sh[j & 1][2] | flag_sh[j & 1][3];  // 1: bad pages, 2: wide
        if constexpr (kQuant) {
          const float* vm = vmax_sh[j & 1];
          const float v = fmaxf(fmaxf(vm[0], vm[1]), fmaxf(vm[2], vm[3]));
          // The unit's reference is at most an 8th of a scale that all rows have seen (seen_by_all), or the least one of the
          // unit's first tile, so that it is nowhere far above what a row has seen.  (That of a tile in which rows differ
          // is a power of two: with which one a row's weights are multiplied, by the scales of keys that it does not see, is
          // then nothing to it.)
          bool wide = false;
          if (piece_first) seen_by_all = 0.f;
          if (mixed) {
            const float* vl = vmin_sh[j & 1];
            const float least = fminf(fminf(vl[0], vl[1]), fminf(vl[2], vl[3]));
            if (piece_first) {
              vref = pow2_at(least < INFINITY ? 0.125f * least : 0.f);
              vinv = pow2_inverse(vref);
            }
            wide = v > kMostFactor * vref || (least < vref && seen_by_all < 8.f * vref);
          } else {
            seen_by_all = fmaxf(seen_by_all, v);
            if (piece_first || v > kMostFactor * vref || seen_by_all < 8.f * vref) {
              vref = scale_reference(seen_by_all);
              vinv = 1.f / vref;
            }
          }
          const float tref = wide ? fminf(pow2_at(v * 0.0625f), kMostRef) : vref;
          ks[lt] = ksv;
          // (a scale that is not finite counts as 0 here; the rows that see it add the products at the end)
          const bool finite = fabsf(vsv) < INFINITY;
          ks[128 + lt] = finite ? vsv * (wide ? pow2_inverse(tref) : vinv) : 0.f;
          if (!finite) poison_sh[unit % G::kRing] = unit + 1;
          if (lt == 0) ks[256 + 5] = tref;
          if (wide) flags |= 2;
        }
        if (lt == 0) badw[4] = flags;
        mbar_arrive(info + 8 * ring);
        const bool mixed_now = mixed;
        const int unit_now = unit;
        if (j + 1 < total) look_up();
        // ---- keys (side 0) and values (side 1)
#pragma unroll 1
        for (int side = 0; side < 2 && ok; ++side) {
          const int idx = 2 * j + side;
          const char* pool = (side ? a.c.v : a.c.k) + ch * 16;
          uint32_t dst;
          if constexpr (kQuant) {
            dst = sbase + G::kOffStage + (idx % BUFS) * G::kStage + lt * 16;
          } else {
            ok = freed(idx);
            if (!ok) break;
            dst = sbase + G::kOffRing + (idx % NS) * G::kTile + put0;
          }
          constexpr int kNext = kQuant ? kLoaders * 16 : kStep * 128;
          if (!kQuant && side == 1 && mixed_now) {
            // values that only some rows see: infinities and NaN become zeros (the rows that see them add them at the end)
            bool found = false;
#pragma unroll 4
            for (int x = 0; x < kCount; ++x) {
              const long long of = o[r0 + x * kStep];
              const uint4 w = of != kNoRow ? __ldg(reinterpret_cast<const uint4*>(pool + of * 2)) : make_uint4(0, 0, 0, 0);
              const uint4 z = make_uint4(finite2<kBF>(w.x), finite2<kBF>(w.y), finite2<kBF>(w.z), finite2<kBF>(w.w));
              found |= z.x != w.x || z.y != w.y || z.z != w.z || z.w != w.w;
              sts128(dst + x * kNext, z);
            }
            if (found) poison_sh[unit_now % G::kRing] = unit_now + 1;
          } else {
#pragma unroll
            for (int x0 = 0; x0 < kCount; x0 += kBatch) {
              long long of[kBatch];
#pragma unroll
              for (int x = 0; x < kBatch; ++x) of[x] = o[r0 + (x0 + x) * kStep];
#pragma unroll
              for (int x = 0; x < kBatch; ++x)
                cp_async16(dst + (x0 + x) * kNext, pool + (of[x] != kNoRow ? of[x] * (kQuant ? 1 : 2) : 0), of[x] != kNoRow ? 16 : 0);
            }
          }
          cp_commit();
          if (said <= idx - G::kLag) {
            cp_wait<G::kLag>();
            if constexpr (kQuant) ok = convert(said++);
            else landed(said++);
          }
        }
      }
      cp_wait<0>();
      while (ok && said < 2 * total) {
        if constexpr (kQuant) ok = convert(said++);
        else landed(said++);
      }
      if (!ok) a.desc[8 * c + 6] = 1;
    }
  }
  // every product has completed: its commits were waited for by the rows' last outputs, or (after an error) here
  __syncthreads();
  if (wid == 12) {
    if (lane == 0) {
      // an extra commit, on a barrier of its own, covers whatever was issued
      mma_commit(1, all_done);
      mbar_wait(all_done, 0);
    }
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int D, int FMT, bool QBF>
cudaError_t launch_one(PagedAttnArgs& a, int num_sms, cudaStream_t st) {
  using G = ChunkGeo<D, FMT>;
  static std::atomic<unsigned long long> done{0};
  const int smem = G::kFixed + (a.rq.n_req + 1) * 8;
  static_assert(G::kFixed + 1025 * 8 + 512 <= 227 * 1024, "shared memory");
  cudaError_t e = set_smem_once(paged_chunk_kernel<D, FMT, QBF>, G::kFixed + 1025 * 8, done);
  if (e != cudaSuccess) return e;
  // the warps' register split needs the launch's 512 x 128
  static const int regs = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, paged_chunk_kernel<D, FMT, QBF>) == cudaSuccess ? f.numRegs : 0;
  }();
  if (regs != 128) return cudaErrorInvalidConfiguration;
  const long long rt = (static_cast<long long>(a.rq.max_new) * a.s.group + kChunkRows - 1) / kChunkRows;
  const long long most = static_cast<long long>(a.rq.n_req) * a.c.n_kv * rt * ((a.rq.max_len + kBN - 1) / kBN + 1);
  a.ctas = static_cast<int>(most < num_sms ? most : num_sms);
  paged_chunk_kernel<D, FMT, QBF><<<a.ctas, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_dim(PagedAttnArgs& a, int fmt, int qtype, int num_sms, cudaStream_t st) {
  const bool bf = qtype == kTBf16;
  switch (fmt) {
    case kKvBf16: return launch_one<D, kKvBf16, true>(a, num_sms, st);
    case kKvF16: return launch_one<D, kKvF16, false>(a, num_sms, st);
    case kKvInt8: return bf ? launch_one<D, kKvInt8, true>(a, num_sms, st) : launch_one<D, kKvInt8, false>(a, num_sms, st);
    default: return bf ? launch_one<D, kKvE4m3, true>(a, num_sms, st) : launch_one<D, kKvE4m3, false>(a, num_sms, st);
  }
}

}  // namespace

cudaError_t launch_paged_chunk(PagedAttnArgs& a, int head_dim, int fmt, int qtype, int num_sms, cudaStream_t st) {
  a.s.rows = kChunkRows;
  a.s.bn = kBN;
  return head_dim == 64 ? launch_dim<64>(a, fmt, qtype, num_sms, st) : launch_dim<128>(a, fmt, qtype, num_sms, st);
}

}  // namespace df2
