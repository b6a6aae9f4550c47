// Pieces that the kernels on the fifth-generation tensor cores for many query rows share: shared memory's layout, matrix
// descriptors, products, tensor memory.
#pragma once

#include "common.cuh"
#include "paged.h"
#include "pipeline.cuh"

namespace df2 {

constexpr int kM = 128;        // rows per tile
constexpr int kLoaders = 128;  // threads that bring keys and values

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

// 64 columns as bits: those below n, and a word whose bit 0 is column n.
DF2_DEV unsigned long long columns_below(int n) { return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull); }
DF2_DEV unsigned long long columns_shifted(unsigned long long w, int n) {
  return n >= 64 || n <= -64 ? 0ull : (n >= 0 ? w << n : w >> -n);
}

}  // namespace df2
