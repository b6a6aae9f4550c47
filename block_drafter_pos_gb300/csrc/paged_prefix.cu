// Attention of a group's query rows over its shared prefix: the kernel for many rows per KV head, on the fifth-generation
// tensor cores.
//
// All rows of a group see all of its prefix, so nothing is masked but the last tile's end and bad pages, and a tile's
// value scales have one reference for all rows.  A unit is 256 rows of one KV head (two tiles of 128) against key tiles of
// 128, with tensor memory, warps and products as in the kernel for prompt chunks; without what that one keeps for rows
// that see different keys, a row's 128 scores stay in registers beside 8-bit caches' scales, too.  The page table is read
// two tiles ahead of the copies.  Units, runs and cut units are dealt and described as there; the partials are joined by a
// launch of their own.  Every wait is bounded.
//
// Measured: 64 tokens of 32 query heads over 32768 bf16 positions of 8 KV heads of 128 (134 MB, 34 GFLOP) 43 us, 3700 clocks a
// tile of 128 keys, of which the products of the two row tiles take 1500 to 1750 each; 11 us pass before the first scores, 4 after the
// last.  48 blocks of 8 over three e4m3 prefixes to 30001 positions (164 GFLOP) 165 us, 1.0 PFLOP/s, 4500 clocks a tile: a row
// tile's softmax takes 2600 there, its scales and value factors 1000 of them.  Under the launch's 128 registers 16-bit caches spill 104
// bytes a thread, 8-bit ones 2.
#include "common.cuh"
#include "paged_mma.cuh"
#include "paged_sched.cuh"
#include "pipeline.cuh"
#include "tensor_memory.cuh"

namespace df2 {
namespace {

using Cursor = PagedCursor<true>;
using pipe::lds128;
using pipe::mbar_arrive;
using pipe::mbar_init_count;
using pipe::mbar_wait;
using pipe::smem_u32;

constexpr int kThreads = 512, kSoft = 256;
constexpr int kLaunchRegs = 128, kSoftRegs = 208, kOtherRegs = 48;
constexpr int kBN = kChunkBn;  // keys per tile
constexpr int kHalf = 64;      // keys whose weights are announced together
constexpr int kAhead = 4;      // tiles whose keys' places are known ahead of their copies
constexpr float kGrow = 8.f;   // log2 of the largest weight

// The chunk kernel's layout, with more tiles of places.
template <int D, int FMT>
struct Geo : ChunkGeo<D, FMT> {
  using G = ChunkGeo<D, FMT>;
  static constexpr int kOffPre = G::kOffOffs + kAhead * 128 * 8;
  static constexpr int kFixed = kOffPre + 1024;
};

// A whole sector (32 bytes, aligned) from a thread, whose row is another line than its neighbours'.
DF2_DEV void store32(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]),
               "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

template <int D, int FMT, bool QBF>
__global__ void __launch_bounds__(kThreads, 1) paged_prefix_kernel(const __grid_constant__ PagedAttnArgs a) {
  using G = Geo<D, FMT>;
  constexpr bool kQuant = G::kQuant;
  constexpr bool kBF = kQuant ? false : QBF;
  constexpr int NS = G::kSlots;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[NS * 2 + G::kRing + 11 + 2 * kAhead];
  __shared__ uint32_t tmem_sh;
  __shared__ int poison_sh[G::kRing];  // by unit: the number (from 1) of the last unit in the slot with a value scale that is not finite
  __shared__ long long tmp[kThreads / 32 + 1];
  static_assert(kSoft * kSoftRegs + (kThreads - kSoft) * kOtherRegs <= kThreads * kLaunchRegs, "the register split");
  const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* const sgen = smem_raw + (sbase - smem_u32(smem_raw));
  const uint32_t full = smem_u32(bars), empty = full + 8 * NS, info = empty + 8 * NS, s_full = info + 8 * G::kRing,
                 p_full = s_full + 16, q_full = p_full + 32, o_done = q_full + 16, all_done = o_done + 16, place_full = all_done + 8,
                 place_free = place_full + 8 * kAhead;
  long long* const pre = reinterpret_cast<long long*>(sgen + G::kOffPre);
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init_count(full + 8 * i, kLoaders);
      mbar_init_count(empty + 8 * i, 1);
    }
    for (int i = 0; i < G::kRing; ++i) {
      mbar_init_count(info + 8 * i, 1);
      poison_sh[i] = 0;
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init_count(s_full + 8 * t, 1);
      mbar_init_count(p_full + 16 * t, 4);
      mbar_init_count(p_full + 16 * t + 8, 4);
      mbar_init_count(q_full + 8 * t, 4);
      mbar_init_count(o_done + 8 * t, 1);
    }
    for (int i = 0; i < kAhead; ++i) {
      mbar_init_count(place_full + 8 * i, 1);
      mbar_init_count(place_free + 8 * i, kLoaders / 32);
    }
    mbar_init_count(all_done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_trigger();
  const long long T = paged_scan<kThreads, true>(a, pre, tmp);
  const long long C = T < gridDim.x ? T : gridDim.x, c = blockIdx.x;
  if (tid == 0) a.desc[8 * c] = -1, a.desc[8 * c + 6] = 0;
  if (c >= C) return;
  const long long t_begin = paged_run_begin(c, C, T), t_end = paged_run_begin(c + 1, C, T);
  // Partials that never come (a wait that gives up) leave NaN in the rows they are joined into; the joining kernel sees to the
  // whole units' rows.
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
  // (One copy of code that runs once: at a launch's start each line of it is fetched from memory.)
  Cursor begin;
  begin.start(a, pre, t_begin, t_end);

  if (wid < 8) {
    // ---------------------------------------------------------------- weights of row tile t
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int t = wid >> 2, lrow = tid & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((wid & 3) * 32) << 16);
    const uint32_t s_col = lane_base + 128 * t, o_col = lane_base + 256 + 128 * t;
    Cursor cc = begin;
    int n = 0, units = 0, gtile = 0, gunit = 0;  // this row tile's key tiles and units so far; the run's
    float m = -INFINITY, l = 0.f, sc = 0.f, vref = 0.f;
    bool active = false;
    // This row's query of the cursor's unit into shared memory (the row tile's scores so far are complete, so its former
    // queries have been read).
    auto enter = [&](const Cursor& u) {
      const int rows = u.n * a.s.group - u.qt * a.s.rows;  // of the unit (may exceed it)
      active = t == 0 || rows > kM;
      if (!active) return;
      const int row = u.qt * a.s.rows + t * kM + lrow;
      const bool valid = t * kM + lrow < rows;
      const int i = row / a.s.group, head = u.h * a.s.group + row % a.s.group;
      const uint4* p = reinterpret_cast<const uint4*>(a.q.p + ((u.b0 + i) * a.q.token_stride + head * a.q.head_stride) * 2);
      // The score's factor stays above 0, so that a masked score stays -infinity: the query takes the scale's sign, and a
      // scale of 0 itself.
      const float sign = a.scale_log2 == 0.f ? 0.f : (a.scale_log2 < 0.f ? -1.f : 1.f);
      sc = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
      float f = 1.f;
      if constexpr (kQuant) {
        float x = 0.f;
#pragma unroll 4
        for (int y = 0; y < D / 8; ++y) {
          const uint4 w = valid ? __ldg(p + y) : make_uint4(0, 0, 0, 0);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = unpack2<QBF>(ww[e]);
            x = fmaxf(x, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        }
        // (to fp16, the codes' exact type: exact from 2^-14 of the row's largest on, off by at most 2^-25 of that below)
        f = pow2_shift(x);
        sc = fmaxf(sc / f, 0x1p-149f);
      }
      const uint32_t q = sbase + t * G::kTile + lrow * 128;
#pragma unroll 4
      for (int x = 0; x < D / 8; ++x) {
        uint4 w = valid ? __ldg(p + x) : make_uint4(0, 0, 0, 0);
        uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (kQuant) {
            const float2 v = unpack2<QBF>(ww[e]);
            ww[e] = pack2<false>(v.x * (f * sign), v.y * (f * sign));
          } else {
            ww[e] = sign == 0.f ? times_zero2<kBF>(ww[e]) : (sign < 0.f ? ww[e] ^ 0x80008000u : ww[e]);
          }
        }
        sts128(q + (x >> 3) * 16384 + (((x & 7) ^ (lrow & 7)) << 4), make_uint4(ww[0], ww[1], ww[2], ww[3]));
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + 8 * t);
    };
    enter(cc);
    while (cc.valid() && ok) {
      const int piece = cc.piece();
      for (int j = 0; active && j < piece; ++j, ++n) {
        // ---- scores of one key tile
        const int tile = gtile + j;
        const int ring = tile % G::kRing;
        const float* ks = reinterpret_cast<const float*>(sgen + G::kOffInfo + ring * G::kInfo);
        const uint32_t* badw = reinterpret_cast<const uint32_t*>(sgen + G::kOffInfo + ring * G::kInfo) + 256;
        // (the scores' products follow the tile's information, whose barrier is then in this use's phase)
        ok = mbar_wait(s_full + 8 * t, static_cast<uint32_t>(n & 1)) &&
             mbar_wait(info + 8 * ring, static_cast<uint32_t>((tile / G::kRing) & 1));
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        fence_after();
        float s[kBN];
#pragma unroll
        for (int x = 0; x < 4; ++x) tm_ld32(s_col + 32 * x, s + 32 * x);
        const int2 fl = *reinterpret_cast<const int2*>(badw + 4);  // whether keys of the tile are not seen; the values' reference
        tm_wait_ld();
        if constexpr (kQuant) {
          const float4* kv = reinterpret_cast<const float4*>(ks);
#pragma unroll
          for (int x = 0; x < kBN; x += 4) {
            const float4 w = kv[x / 4];
            const float2 y0 = mul2(make_float2(s[x], s[x + 1]), make_float2(w.x, w.y));
            const float2 y1 = mul2(make_float2(s[x + 2], s[x + 3]), make_float2(w.z, w.w));
            s[x] = y0.x, s[x + 1] = y0.y, s[x + 2] = y1.x, s[x + 3] = y1.y;
          }
        }
        if (fl.x) {  // bits of the keys that are not seen
          const uint4 w = *reinterpret_cast<const uint4*>(badw);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int x = 0; x < kBN; ++x) s[x] = (ww[x >> 5] >> (x & 31)) & 1u ? -INFINITY : s[x];
        }
        float x0 = s[0], x1 = s[1], x2 = s[2], x3 = s[3];
#pragma unroll
        for (int x = 4; x < kBN - 4; x += 8) {
          x0 = fmaxf(fmaxf(x0, s[x]), s[x + 4]);
          x1 = fmaxf(fmaxf(x1, s[x + 1]), s[x + 5]);
          x2 = fmaxf(fmaxf(x2, s[x + 2]), s[x + 6]);
          x3 = fmaxf(fmaxf(x3, s[x + 3]), s[x + 7]);
        }
        x0 = fmaxf(fmaxf(x0, s[kBN - 4]), x2);
        x1 = fmaxf(fmaxf(x1, s[kBN - 3]), x3);
        const float mx = fmaxf(fmaxf(fmaxf(x0, s[kBN - 2]), s[kBN - 1]), x1) * sc;
        float f = 1.f;  // O's factor
        if (j == 0) {
          m = mx;
        } else if (mx > m + kGrow) {
          f = ex2(m - mx);
          m = mx;
          l *= f;
        }
        if constexpr (kQuant) {  // the values' scales are relative to the tile's reference, and so is O
          const float tref = __int_as_float(fl.y);
          if (j == 0) vref = tref;
          else if (vref != tref) f *= vref * reciprocal(tref);
          vref = tref;
        }
        if (__any_sync(0xffffffffu, f != 1.f)) {  // (the former tile's products came before this one's scores)
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
        // ---- weights (a row that has seen nothing: 2^(-infinity)), announced by halves, summed in fp32 and rounded once, to
        // the product's operand type, which has to be the values'
        const float mr = m == -INFINITY ? 0.f : -m;
        float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
        const float2 sc2 = make_float2(sc, sc), mr2 = make_float2(mr, mr);
        const float4* vv = reinterpret_cast<const float4*>(ks + 128);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[kHalf / 2];
#pragma unroll
          for (int y = 0; y < kHalf; y += 4) {
            const int x = kHalf * h + y;
            float2 a0 = fma2(make_float2(s[x], s[x + 1]), sc2, mr2), a1 = fma2(make_float2(s[x + 2], s[x + 3]), sc2, mr2);
            a0 = make_float2(ex2(a0.x), ex2(a0.y));
            a1 = make_float2(ex2(a1.x), ex2(a1.y));
            acc0 = add2(acc0, a0);
            acc1 = add2(acc1, a1);
            if constexpr (kQuant) {
              const float4 w = vv[x / 4];
              a0 = mul2(a0, make_float2(w.x, w.y));
              a1 = mul2(a1, make_float2(w.z, w.w));
            }
            p[y / 2] = pack2<kBF>(a0.x, a0.y);
            p[y / 2 + 1] = pack2<kBF>(a1.x, a1.y);
          }
          tm_st32(s_col + (kHalf / 2) * h, p);
          tm_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 8 * (2 * t + h));
        }
        acc0 = add2(acc0, acc1);
        l += acc0.x + acc0.y;
      }
      if (!ok) break;
      // ---- the end of the unit (or of the run): the next unit's queries first, then this one's outputs
      Cursor nc = cc;
      nc.skip(a, piece);
      {
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
            dd[7] = 0;
            dd[0] = cc.r;
          }
          ok = mbar_wait(o_done + 8 * t, static_cast<uint32_t>(units++ & 1));  // (of a unit's last products)
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          fence_after();
          const int lr = t * kM + lrow, row = cc.qt * a.s.rows + lr;
          const bool valid = lr < rows;
          const int i = row / a.s.group, head = cc.h * a.s.group + row % a.s.group;
          float* pp = a.part + slot * (a.s.rows * (D + 2)) + lr * D;
          float2* ps = reinterpret_cast<float2*>(a.part + slot * (a.s.rows * (D + 2)) + a.s.rows * D + 2 * lr);
          if (whole && valid) {
            pp = joint_row<D>(a, cc.b0 + i, head);
            ps = joint_stat<D>(a, cc.b0 + i, head);
          }
          const float out_f = kQuant ? vref : 1.f;
          const bool poison = kQuant && *static_cast<volatile int*>(&poison_sh[gunit % G::kRing]) > gunit;
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            float o[32];
            __syncwarp();
            tm_ld32(o_col + 32 * x, o);
            tm_wait_ld();
            if constexpr (kQuant) {
              if (poison && valid) {
                // value scales that are not finite: the product had zeros there
                const int first_i = cc.unit_t >= t_begin ? 0 : static_cast<int>(t_begin - cc.unit_t);
                const int k0 = (cc.u.t0 + first_i) * kBN, k1 = min((cc.u.t0 + i_last + 1) * kBN, cc.len);
                for (int key = k0; key < k1; ++key) {
                  const int page = __ldg(a.c.table + cc.table_row(key) * a.c.table_stride + key / a.c.page_size);
                  long long off, so;
                  if (!paged_row(a.c, page, key % a.c.page_size, cc.h, &off, &so)) continue;
                  const float vs = __ldg(a.c.v_scale + so);
                  if (fabsf(vs) < INFINITY) continue;
                  const uint32_t* v = reinterpret_cast<const uint32_t*>(a.c.v + off + 32 * x);
#pragma unroll
                  for (int y = 0; y < 8; ++y) {
                    const uint32_t w = __ldg(v + y);
                    const float2 v0 = unpack2<false>(codes2<FMT, 0>(w)), v1 = unpack2<false>(codes2<FMT, 1>(w));
                    o[4 * y] += v0.x * vs, o[4 * y + 1] += v0.y * vs, o[4 * y + 2] += v1.x * vs, o[4 * y + 3] += v1.y * vs;
                  }
                }
              }
            }
            if (valid) {
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] *= out_f;
#pragma unroll
              for (int y = 0; y < 32; y += 8) store32(pp + 32 * x + y, o + y);
            }
          }
          if (valid) *ps = make_float2(m, l);
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
      Cursor cs = begin;
      uint32_t fine = 1, units1 = 0, units0 = 0, n0 = 0, n1 = 0;  // units and key tiles of the row tiles so far
      int g = 0;                                                  // key tiles before the unit's
      int last = 0;                                               // its key tiles
      bool two = false;
      // scores of row tile t in the unit's key tile j
      auto scores = [&](uint32_t t, int j) {
        const uint32_t idx = 2 * (g + j), slot = idx % NS;
        if (t == 0) fine &= mbar_wait_warp(full + 8 * slot, (idx / NS) & 1);
        fence_after();
        const uint32_t q = desc_k(sbase + t * G::kTile), kd = desc_k(sbase + G::kOffRing + slot * G::kTile);
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          mma_ss(go, tmem + 128 * t, q + (x >> 2) * 1024 + 2 * (x & 3), kd + (x >> 2) * 1024 + 2 * (x & 3), id_s, x != 0);
        mma_commit(go, s_full + 8 * t);
        if (t == 1 || !two) mma_commit(go, empty + 8 * slot);
      };
      auto outputs = [&](uint32_t t, int j) {
        const uint32_t idx = 2 * (g + j) + 1, slot = idx % NS;
        if (t == 0) fine &= mbar_wait_warp(full + 8 * slot, (idx / NS) & 1);
        const uint32_t ph = (t ? n1 : n0) & 1;
        fine &= mbar_wait_warp(p_full + 16 * t, ph);
        fence_after();
        const uint32_t v = desc_mn(sbase + G::kOffRing + slot * G::kTile), p = tmem + 128 * t, o = tmem + 256 + 128 * t;
#pragma unroll
        for (int x = 0; x < kBN / 32; ++x) mma_ts(go, o, p + 8 * x, v + 128 * x, id_o, x != 0 || j != 0);
        fine &= mbar_wait_warp(p_full + 16 * t + 8, ph);
        fence_after();
#pragma unroll
        for (int x = kBN / 32; x < kBN / 16; ++x) mma_ts(go, o, p + 8 * x, v + 128 * x, id_o, 1);
        if (j + 1 == last) mma_commit(go & fine, o_done + 8 * t);
        if (t == 1 || !two) mma_commit(go, empty + 8 * slot);
        if (t) ++n1;
        else ++n0;
      };
      // (a failed wait ends the loop at the tile's end, and no output is announced after it: the others' waits run out in turn)
      while (cs.valid() && fine) {
        const int piece = cs.piece();
        last = piece;
        two = __any_sync(0xffffffffu, cs.n * a.s.group - cs.qt * a.s.rows > kM);
        fine &= mbar_wait_warp(q_full, units0 & 1);
        if (two) fine &= mbar_wait_warp(q_full + 8, units1 & 1);
        ++units0;
        if (two) ++units1;
        for (int j = -1; j < piece; ++j) {
#pragma unroll 1
          for (uint32_t t = 0; t < (two ? 2u : 1u); ++t) {
            if (j >= 0) outputs(t, j);
            if (j + 1 < piece) scores(t, j + 1);
          }
          if (!__all_sync(0xffffffffu, fine != 0)) {
            fine = 0;
            break;
          }
        }
        g += piece;
        cs.skip(a, piece);
      }
      ok = fine != 0;
      if (!ok && lane == 0) a.desc[8 * c + 6] = 1;
    } else if (wid == 13) {
      // -------------------------------------------------------------- places and scales of a tile's keys, four a lane
      // The page table is read two tiles, the scales one tile before they are handed on, so that no latency of theirs is on the
      // way, and all of it by this warp ahead of the loaders (in their loop it took as long as the copies and conversions: 48
      // blocks over e4m3 prefixes of 30001 positions 316 us, 292 so).
      long long* const offs = reinterpret_cast<long long*>(sgen + G::kOffOffs);
      Cursor lc = begin;
      const int total = static_cast<int>(t_end - t_begin);
      int page[4], row[4];  // of the tile fetched last; row -1: no key of the prefix
      int pg_h = 0, pg_r = 0, unit = 0;
      bool pg_first = true, l_first = true, piece_first = true;
      long long off[4];
      float ksv[4], vsv[4];
      uint32_t unseen = 0;
      auto fetch = [&]() {
        if (!lc.valid()) return;
        const int key0 = (lc.u.t0 + lc.i) * kBN + 4 * lane;
        pg_first = l_first;
        pg_h = lc.h;
        pg_r = lc.r;
        int pi = key0 / a.c.page_size, x = key0 - pi * a.c.page_size;
        const int32_t* const table = a.c.table + lc.table_row(key0) * a.c.table_stride;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          row[e] = key0 + e < lc.u.hi ? x : -1;
          if (row[e] >= 0) page[e] = __ldg(table + pi);
          if (++x == a.c.page_size) x = 0, ++pi;
        }
        l_first = lc.unit_ends();
        lc.next(a);
      };
      auto resolve = [&]() {
        piece_first = pg_first;
        unseen = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          off[e] = kNoRow;
          ksv[e] = vsv[e] = 0.f;
          long long o, so;
          if (row[e] >= 0 && paged_row(a.c, page[e], row[e], pg_h, &o, &so)) {
            off[e] = o;
            if (kQuant) {
              ksv[e] = __ldg(a.c.k_scale + so);
              vsv[e] = __ldg(a.c.v_scale + so);
            }
          } else {
            unseen |= 1u << e;
            if (row[e] >= 0) paged_flag<true>(a, pg_r, 1);  // DFLASH2_E_INVAL
          }
        }
      };
      float vref = 0.f, vinv = 0.f, largest = 0.f;
      for (int step = 0; step < total + 2; ++step) {
        if (step >= 2) {  // hand on tile j
          const int j = step - 2;
          const int ring = j % G::kRing, slot = j % kAhead;
          float* ks = reinterpret_cast<float*>(sgen + G::kOffInfo + ring * G::kInfo);
          uint32_t* badw = reinterpret_cast<uint32_t*>(ks + 256);
          if (piece_first && j > 0) ++unit;
          // (The loaders have copied tile j - 4, so operands up to that of tile j - 7 have been read, and the weights of the tile
          // that had this slot of the information, eight ago, are done.)
          ok = j < kAhead || mbar_wait(place_free + 8 * slot, static_cast<uint32_t>((j / kAhead + 1) & 1));
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          if constexpr (kQuant) {
            // A 16th of the largest scale so far, raised when one exceeds 128 of it, so that fp16 holds a weight (at most 2^8)
            // times a scale over it
            float v = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) v = vsv[e] < INFINITY ? fmaxf(v, vsv[e]) : v;
            v = warp_max(v);
            if (piece_first) largest = 0.f;
            largest = fmaxf(largest, v);
            if (piece_first || v > kMostFactor * vref || largest < 8.f * vref) {
              vref = scale_reference(largest);
              vinv = 1.f / vref;
            }
            // (a scale that is not finite counts as 0 here; its products are added at the end)
            float vf[4];
            bool finite = true;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool fine = fabsf(vsv[e]) < INFINITY;
              vf[e] = fine ? vsv[e] * vinv : 0.f;
              finite = finite && fine;
            }
            if (!finite) poison_sh[unit % G::kRing] = unit + 1;
            reinterpret_cast<float4*>(ks)[lane] = make_float4(ksv[0], ksv[1], ksv[2], ksv[3]);
            reinterpret_cast<float4*>(ks + 128)[lane] = make_float4(vf[0], vf[1], vf[2], vf[3]);
            if (lane == 0) ks[256 + 5] = vref;
          }
          const bool any = __any_sync(0xffffffffu, unseen != 0);
          if (any) {
            uint32_t w = unseen << (4 * (lane & 7));
#pragma unroll
            for (int x = 1; x <= 4; x <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, x);
            if ((lane & 7) == 0) badw[lane >> 3] = w;
          }
          if (lane == 0) badw[4] = any ? 1u : 0u;
          long long* const o = offs + slot * 128 + 4 * lane;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = off[e];
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(info + 8 * ring);
            mbar_arrive(place_full + 8 * slot);
          }
        }
        if (step >= 1 && step <= total) resolve();
        if (step < total) fetch();
      }
      if (!ok && lane == 0) a.desc[8 * c + 6] = 1;
    } else if (wid < 12) {
      // -------------------------------------------------------------- keys and values
      const int lt = tid - kSoft;
      const int total = static_cast<int>(t_end - t_begin);
      // A thread copies piece ch of rows r0, r0 + kApart, ...: the swizzle's row bits are its own constant.
      constexpr int kPieces = D * (kQuant ? 1 : 2) / 16, kApart = kLoaders / kPieces, kCount = 128 / kApart;
      constexpr int kBatch = kCount < 8 ? kCount : 8, BUFS = G::kBufs > 0 ? G::kBufs : 1;
      const int ch = lt % kPieces, r0 = lt / kPieces;
      // where piece ch of row r0 goes (16-bit: itself; codes: the first of its two pieces of fp16)
      const int piece = kQuant ? 2 * ch : ch;
      const uint32_t put0 = (piece >> 3) * 16384 + r0 * 128 + (((piece & 7) ^ (r0 & 7)) << 4);
      const uint32_t put1 = (piece >> 3) * 16384 + r0 * 128 + ((((piece & 7) + 1) ^ (r0 & 7)) << 4);
      static_assert(kApart % 8 == 0, "a thread's rows share their place in the swizzle");
      auto landed = [&](int idx) {  // this thread's part of operand idx is in place
        fence_async();
        mbar_arrive(full + 8 * (idx % NS));
      };
      auto freed = [&](int idx) {  // the operand that had idx's slot has been read
        const int use = idx / NS;
        return use == 0 || mbar_wait(empty + 8 * (idx % NS), static_cast<uint32_t>((use + 1) & 1));
      };
      // 8-bit: this thread's codes of operand idx from the staging area to its slot
      auto convert = [&](int idx) {
        if (!freed(idx)) return false;
        if constexpr (kQuant) {
          const uint32_t st = sbase + G::kOffStage + (idx % BUFS) * G::kStage + lt * 16;
          const uint32_t dst = sbase + G::kOffRing + (idx % NS) * G::kTile;
#pragma unroll
          for (int x0 = 0; x0 < kCount; x0 += 4) {
            uint4 w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] = lds128(st + (x0 + x) * (kLoaders * 16));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t d = dst + (x0 + x) * (kApart * 128);
              sts128(d + put0, make_uint4(codes2<FMT, 0>(w[x].x), codes2<FMT, 1>(w[x].x), codes2<FMT, 0>(w[x].y), codes2<FMT, 1>(w[x].y)));
              sts128(d + put1, make_uint4(codes2<FMT, 0>(w[x].z), codes2<FMT, 1>(w[x].z), codes2<FMT, 0>(w[x].w), codes2<FMT, 1>(w[x].w)));
            }
          }
        }
        landed(idx);
        return true;
      };
      int said = 0;  // operands announced
      for (int j = 0; j < total && ok; ++j) {
        const int slot = j % kAhead;
        const long long* const o = reinterpret_cast<const long long*>(sgen + G::kOffOffs) + slot * 128 + r0;
        ok = __all_sync(0xffffffffu, mbar_wait(place_full + 8 * slot, static_cast<uint32_t>((j / kAhead) & 1)));  // (the warp ends as one)
        // ---- keys (side 0) and values (side 1)
#pragma unroll 1
        for (int side = 0; side < 2 && ok; ++side) {
          const int idx = 2 * j + side;
          const char* pool = (side ? a.c.v : a.c.k) + ch * 16;
          uint32_t dst;
          if constexpr (kQuant) {
            dst = sbase + G::kOffStage + (idx % BUFS) * G::kStage + lt * 16;
          } else {
            ok = __all_sync(0xffffffffu, freed(idx));
            if (!ok) break;
            dst = sbase + G::kOffRing + (idx % NS) * G::kTile + put0;
          }
          constexpr int kNext = kQuant ? kLoaders * 16 : kApart * 128;
#pragma unroll
          for (int x0 = 0; x0 < kCount; x0 += kBatch) {
            long long of[kBatch];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) of[x] = o[(x0 + x) * kApart];
#pragma unroll
            for (int x = 0; x < kBatch; ++x)
              cp_async16(dst + (x0 + x) * kNext, pool + (of[x] != kNoRow ? of[x] * (kQuant ? 1 : 2) : 0), of[x] != kNoRow ? 16 : 0);
          }
          cp_commit();
          if (side == 1) {  // (the tile's places have been read)
            __syncwarp();
            if (lane == 0) mbar_arrive(place_free + 8 * slot);
          }
          if (said <= idx - G::kLag) {
            cp_wait<G::kLag>();
            if constexpr (kQuant) ok = __all_sync(0xffffffffu, convert(said++));
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
  using G = Geo<D, FMT>;
  static std::atomic<unsigned long long> done{0};
  const int smem = G::kFixed + (a.rq.n_req + 1) * 8;
  cudaError_t e = set_smem_once(paged_prefix_kernel<D, FMT, QBF>, G::kFixed + 1025 * 8, done);
  if (e != cudaSuccess) return e;
  // the warps' register split needs the launch's 512 x 128
  static const int regs = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, paged_prefix_kernel<D, FMT, QBF>) == cudaSuccess ? f.numRegs : 0;
  }();
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  const long long rt = (static_cast<long long>(a.rq.max_new) * a.s.group + kChunkRows - 1) / kChunkRows;
  const long long most = static_cast<long long>(a.rq.n_req) * a.c.n_kv * rt * ((a.rq.max_len + kBN - 1) / kBN + 1);
  a.ctas = static_cast<int>(most < num_sms ? most : num_sms);
  paged_prefix_kernel<D, FMT, QBF><<<a.ctas, kThreads, smem, st>>>(a);
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

cudaError_t launch_shared_prefix(PagedAttnArgs& a, int head_dim, int fmt, int qtype, int num_sms, cudaStream_t st) {
  a.s.rows = kChunkRows;
  a.s.bn = kBN;
  return head_dim == 64 ? launch_dim<64>(a, fmt, qtype, num_sms, st) : launch_dim<128>(a, fmt, qtype, num_sms, st);
}

}  // namespace df2
