// Pieces that the paged attention's kernels share.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.h"

namespace df2 {

DF2_DEV uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
DF2_DEV void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
DF2_DEV void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
DF2_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
DF2_DEV void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
DF2_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF>
DF2_DEV uint32_t pack2(float lo, float hi) {
  if constexpr (BF) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
template <bool BF>
DF2_DEV float2 unpack2(uint32_t w) {
  if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Two 16-bit values with zeros in the place of infinities and NaN.
template <bool BF>
DF2_DEV uint32_t finite2(uint32_t w) {
  constexpr uint32_t ex = BF ? 0x7F80u : 0x7C00u;
  if ((w & ex) == ex) w &= 0xFFFF0000u;
  if (((w >> 16) & ex) == ex) w &= 0x0000FFFFu;
  return w;
}

// Two 16-bit values times zero: NaN for infinities and NaN.
template <bool BF>
DF2_DEV uint32_t times_zero2(uint32_t w) {
  constexpr uint32_t ex = BF ? 0x7F80u : 0x7C00u;
  return ((w & ex) == ex ? 0x7FFFu : 0u) | (((w >> 16) & ex) == ex ? 0x7FFF0000u : 0u);
}

// Two fp32 values at a time (the packed fp32 instructions of this architecture).
DF2_DEV float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}
DF2_DEV float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
DF2_DEV float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}

// Two codes (bytes 0, 1 or 2, 3 of w) as exact fp16 values.
template <int FMT, int HI>
DF2_DEV uint32_t codes2(uint32_t w) {
  if constexpr (FMT == kKvInt8) {
    return codes_to_half2(w ^ 0x80808080u, HI ? 0x4342u : 0x4140u);
  } else {
    uint32_t h;
    if constexpr (HI) asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %1;\n cvt.rn.f16x2.e4m3x2 %0, y;\n}\n" : "=r"(h) : "r"(w));
    else asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %1;\n cvt.rn.f16x2.e4m3x2 %0, x;\n}\n" : "=r"(h) : "r"(w));
    return h;
  }
}

// Ones in the bytes of w that are e4m3 codes of NaN (0x7F and 0xFF).
DF2_DEV uint32_t nan_codes(uint32_t w) { return ((((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu; }

// 2^-e with x in [2^e, 2^(e + 1)); 1 for zero, tiny and nonfinite x.  Rows of queries are brought to
// fp16's range with it, exactly.
DF2_DEV float pow2_shift(float x) {
  const uint32_t ex = __float_as_uint(x) >> 23;
  return ex == 0 || ex >= 254 ? 1.f : __uint_as_float((254u - ex) << 23);
}

// The values' reference: weights of an 8-bit cache (at most 2^8) are multiplied by their value's scale relative to it.  It
// begins at a 16th of a scale (whose value then has a factor of 16) and is raised when one exceeds 128 of it: so far up
// fp16 holds the product, and down to 2^-25 of the largest scale or less it tells weights apart.  Within [2^-126, 2^126], so that its
// reciprocal is a normal number.
constexpr float kMostFactor = 128.f;
DF2_DEV float in_reference_range(float x) { return fminf(fmaxf(x, 0x1p-126f), 0x1p126f); }
DF2_DEV float scale_reference(float v) { return in_reference_range(v * 0.0625f); }
DF2_DEV float reciprocal(float x) {  // within 2^-23
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The power of two at x, within [2^-126, 2^126], and its exact reciprocal and exponent.
DF2_DEV float pow2_at(float x) { return __uint_as_float(__float_as_uint(in_reference_range(x)) & 0x7F800000u); }
DF2_DEV float pow2_inverse(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }
DF2_DEV float pow2_exponent(float x) { return static_cast<float>(static_cast<int>(__float_as_uint(x) >> 23) - 127); }

}  // namespace df2
