// Writing keys and values into the paged cache and reading them back.
//
// Quantised formats: s = max(amax|x| / Q, 2^-126) per (position, KV head) and side, code =
// x / s rounded to nearest even and saturated, value = code * s.  Both divisions are IEEE
// (so a code never depends on how a reciprocal rounds), and |x / s| <= Q up to one rounding.
//
// Both directions are streams: a warp per token, 8 channels per lane and load, the keys' and
// the values' loads issued together, amax by shuffles within the row's lanes, so each source
// element is read once and each code written once.  Measured for 40,005 tokens of 8 heads of 128 (248 MB each
// way): bf16 to e4m3 68 us (3.6 TB/s: instruction issue, 2.8 of 4 a clock, about 175 for 8 channels of a lane), back to
// bf16 41 us (6.0 TB/s, 89% of a copy's rate).  From bf16 to a bf16 or fp16 pool (328 MB) 53 us, 6.2 TB/s, from fp32
// (492 MB) 75, 6.6 TB/s; from fp32 to int8 or e4m3 (412 MB) 70 and 67.
#include "common.cuh"
#include "paged.h"
#include "paged_mma.cuh"

namespace df2 {
namespace {

constexpr int kThreads = 256;

// Whether request r can be served: its range and its length are within bounds, and its new tokens within its length.
DF2_DEV bool good_request(const PagedReq& q, int r, int& b0, int& b1, int& len) {
  b0 = __ldg(q.begin + r), b1 = __ldg(q.begin + r + 1), len = __ldg(q.kv_len + r);
  return paged_request_ok(q, b0, b1, len) && len >= b1 - b0;
}

// The first block flags the requests that cannot be served.
DF2_DEV void flag_requests(const PagedReq& q) {
  if (blockIdx.x != 0 || !q.status) return;
  int b0, b1, len;
  for (int r = threadIdx.x; r < q.n_req; r += kThreads)
    if (!good_request(q, r, b0, b1, len)) q.status[r] = 1;  // DFLASH2_E_INVAL
}

// Request of packed row t and the row's position in its cache; false if no good request holds the row.  A whole warp
// calls it for one row.
DF2_DEV bool find_position(const PagedReq& q, int t, int& r, int& pos) {
  int lo = 0, hi = q.n_req;  // the last r with begin[r] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(q.begin + mid) <= t) lo = mid;
    else hi = mid;
  }
  int b0, b1, len;
  r = lo;
  if (!good_request(q, r, b0, b1, len) || t < b0 || t >= b1) {
    // a bad range may have misled the search: the first good request that holds the row
    const int lane = threadIdx.x & 31;
    uint32_t m = 0;
    int r0 = -32;
    while (m == 0 && (r0 += 32) < q.n_req) {
      r = r0 + lane;
      m = __ballot_sync(0xffffffffu, r < q.n_req && good_request(q, r, b0, b1, len) && t >= b0 && t < b1);
    }
    if (m == 0) return false;
    r = r0 + __ffs(m) - 1;
    good_request(q, r, b0, b1, len);
  }
  pos = len - (b1 - b0) + (t - b0);
  return true;
}

// Element offsets of (request r, position pos, KV head h) in the pools and the scales.
DF2_DEV bool find_row(const PagedCache& c, const PagedReq& q, int r, int pos, int h, long long& off, long long& soff) {
  const int page_i = pos / c.page_size, row = pos - page_i * c.page_size;
  const int page = __ldg(c.table + r * c.table_stride + page_i);
  if (paged_row(c, page, row, h, &off, &soff)) return true;
  if (q.status) q.status[r] = 1;
  return false;
}

template <int T>
DF2_DEV void load8(const char* p, long long off, float (&x)[8]) {
  if constexpr (T == kTF32) {
    const float4* s = reinterpret_cast<const float4*>(p + off * 4);
    const float4 a = s[0], b = s[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p + off * 2);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (T == kTBf16) f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      else f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
}

template <int T>
DF2_DEV void store8(char* p, long long off, const float (&x)[8]) {
  if constexpr (T == kTF32) {
    float4* s = reinterpret_cast<float4*>(p + off * 4);
    s[0] = make_float4(x[0], x[1], x[2], x[3]);
    s[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T == kTBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    *reinterpret_cast<uint4*>(p + off * 2) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// |x| of 8 values as bits, the largest: ordered as the values are, infinity above every number and NaN above
// infinity, so a nonfinite element always wins.
template <int T>
DF2_DEV uint32_t largest8(const float (&x)[8]) {
  if constexpr (T == kTBf16) {  // two to a word, as they came
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632) & 0x7FFF7FFFu;
      asm("max.u16x2 %0, %0, %1;" : "+r"(m2) : "r"(w));
    }
    return max(m2 << 16, m2 & 0xFFFF0000u);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return m;
}

// Codes of 8 channels: x / s, IEEE-rounded, then rounded to nearest even and saturated.  x (1 / s) (1 +- 2^-21) bound that
// quotient from both sides, and rounding to a code is monotonic: where both give one code it is the quotient's, and
// only where they differ (a few in 100,000) is the division done.  (16 divisions a thread made the kernel issue-bound.)
template <int FMT>
DF2_DEV uint2 codes8(const float (&x)[8], float s) {
  float inv;  // within 2^-23; s is at least 2^-126
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const float up = inv * 1.000000476837158f, down = inv * 0.999999523162842f;
  const float2 up2 = make_float2(up, up), down2 = make_float2(down, down);
  uint32_t w[2] = {0u, 0u}, differ = 0u;
  if constexpr (FMT == kKvInt8) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the rounded integer
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 y = make_float2(x[i], x[i + 1]);
      const float2 u = fma2(y, up2, make_float2(kMagic, kMagic)), d = fma2(y, down2, make_float2(kMagic, kMagic));
      c[i] = __float_as_uint(u.x), c[i + 1] = __float_as_uint(u.y);
      differ |= (c[i] ^ __float_as_uint(d.x)) | (c[i + 1] ^ __float_as_uint(d.y));
    }
    if (differ) {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = __float_as_uint(__fdiv_rn(x[i], s) + kMagic);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
  } else {
    auto pair = [](float lo, float hi) {
      uint16_t c;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
      return static_cast<uint32_t>(c);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = make_float2(x[2 * i], x[2 * i + 1]), u = mul2(y, up2), d = mul2(y, down2);
      const uint32_t c = pair(u.x, u.y);
      differ |= c ^ pair(d.x, d.y);
      w[i >> 1] |= c << (16 * (i & 1));
    }
    if (differ) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = pair(__fdiv_rn(x[4 * i], s), __fdiv_rn(x[4 * i + 1], s)) | (pair(__fdiv_rn(x[4 * i + 2], s), __fdiv_rn(x[4 * i + 3], s)) << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}

// A warp moves one token: its position is found once, and lane l takes pieces l, l + 32, ... of 8 channels of its
// heads' rows (a row's D / 8 lanes are neighbours), two at a time so that four loads are in flight.
template <int D, int FMT, int T>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ PagedMoveArgs a) {
  constexpr int kLanes = D / 8;  // of a row
  const int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  flag_requests(a.rq);
  if (t >= a.rq.n_tokens) return;
  const char* const pk = a.k.p + t * a.k.token_stride * (T == kTF32 ? 4 : 2);
  const char* const pv = a.v.p + t * a.v.token_stride * (T == kTF32 ? 4 : 2);
  const int pieces = a.c.n_kv * kLanes;
  int r, pos;
  long long off, soff;
  const bool go = find_position(a.rq, t, r, pos) && find_row(a.c, a.rq, r, pos, 0, off, soff);
  if (!go) return;  // (the whole warp)
  for (int p0 = 0; p0 < pieces; p0 += 64) {
    float x[2][2][8];
    int h[2];
    const int ch = (lane % kLanes) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = p0 + 32 * i + lane;
      h[i] = p < pieces ? p / kLanes : 0;  // (idle lanes redo head 0 and store nothing)
      load8<T>(pk, h[i] * a.k.head_stride + ch, x[i][0]);
      load8<T>(pv, h[i] * a.v.head_stride + ch, x[i][1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = p0 + 32 * i + lane < pieces;
      const long long o = off + h[i] * a.c.head_stride + ch, so = soff + h[i] * a.c.s_head_stride;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        char* const pool = side ? a.c.v : a.c.k;
        if constexpr (FMT == kKvBf16 || FMT == kKvF16) {
          if (in) store8<FMT == kKvBf16 ? kTBf16 : kTF16>(pool, o, x[i][side]);
        } else {
          uint32_t m = largest8<T>(x[i][side]);
#pragma unroll
          for (int of = kLanes / 2; of > 0; of >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, of));
          const bool fine = m < 0x7F800000u;
          float s = __fdiv_rn(__uint_as_float(m), FMT == kKvInt8 ? 127.f : 448.f);
          if (fine) s = fmaxf(s, 1.17549435e-38f);  // 2^-126
          uint2 w = codes8<FMT>(x[i][side], s);
          if (!fine) w = make_uint2(0u, 0u);
          if (in) {
            *reinterpret_cast<uint2*>(pool + o) = w;
            if (ch == 0) (side ? a.c.v_scale : a.c.k_scale)[so] = s;
          }
        }
      }
    }
  }
}

template <int FMT>
struct Raw8 {  // 8 channels as the pool holds them
  uint4 w;
  float s;
  DF2_DEV void load(const char* pool, const float* scales, long long off, long long soff) {
    if constexpr (FMT == kKvBf16 || FMT == kKvF16) {
      w = *reinterpret_cast<const uint4*>(pool + off * 2);
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(pool + off);
      w.x = v.x, w.y = v.y;
      s = scales[soff];
    }
  }
  DF2_DEV void values(float (&x)[8]) const {
    if constexpr (FMT == kKvBf16 || FMT == kKvF16) {
      const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c = unpack2<FMT == kKvBf16>(p[i]);
        x[2 * i] = c.x, x[2 * i + 1] = c.y;
      }
    } else {
      const uint32_t p[4] = {codes2<FMT, 0>(w.x), codes2<FMT, 1>(w.x), codes2<FMT, 0>(w.y), codes2<FMT, 1>(w.y)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c = unpack2<false>(p[i]);  // (exact)
        x[2 * i] = c.x * s, x[2 * i + 1] = c.y * s;
      }
    }
  }
};

template <int D, int FMT, int T>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ PagedMoveArgs a) {
  constexpr int kLanes = D / 8;
  const int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  flag_requests(a.rq);
  if (t >= a.rq.n_tokens) return;
  int r, pos;
  if (!find_position(a.rq, t, r, pos)) return;
  long long off = 0, soff = 0;
  const bool good = find_row(a.c, a.rq, r, pos, 0, off, soff);
  char* const pk = a.k.p + t * a.k.token_stride * (T == kTF32 ? 4 : 2);
  char* const pv = a.v.p + t * a.v.token_stride * (T == kTF32 ? 4 : 2);
  const int pieces = a.c.n_kv * kLanes, ch = (lane % kLanes) * 8;
  for (int p0 = lane; p0 < pieces; p0 += 128) {
    Raw8<FMT> k[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = (p0 + 32 * i) / kLanes;
      if (good && p0 + 32 * i < pieces) {
        k[i].load(a.c.k, a.c.k_scale, off + h * a.c.head_stride + ch, soff + h * a.c.s_head_stride);
        v[i].load(a.c.v, a.c.v_scale, off + h * a.c.head_stride + ch, soff + h * a.c.s_head_stride);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = (p0 + 32 * i) / kLanes;
      if (p0 + 32 * i >= pieces) break;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (good) k[i].values(x);
      store8<T>(pk, h * a.k.head_stride + ch, x);
      if (good) v[i].values(x);
      store8<T>(pv, h * a.v.head_stride + ch, x);
    }
  }
}

template <int D, int FMT>
cudaError_t launch_move(const PagedMoveArgs& a, bool write, cudaStream_t st) {
  constexpr int kTokens = kThreads / 32;  // of a block
  const dim3 grid((a.rq.n_tokens + kTokens - 1) / kTokens);
  switch (a.k.type * 2 + (write ? 1 : 0)) {
    case kTBf16 * 2 + 1: write_kernel<D, FMT, kTBf16><<<grid, kThreads, 0, st>>>(a); break;
    case kTF16 * 2 + 1: write_kernel<D, FMT, kTF16><<<grid, kThreads, 0, st>>>(a); break;
    case kTF32 * 2 + 1: write_kernel<D, FMT, kTF32><<<grid, kThreads, 0, st>>>(a); break;
    case kTBf16 * 2: read_kernel<D, FMT, kTBf16><<<grid, kThreads, 0, st>>>(a); break;
    case kTF16 * 2: read_kernel<D, FMT, kTF16><<<grid, kThreads, 0, st>>>(a); break;
    default: read_kernel<D, FMT, kTF32><<<grid, kThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_move_fmt(const PagedMoveArgs& a, int fmt, bool write, cudaStream_t st) {
  switch (fmt) {
    case kKvBf16: return launch_move<D, kKvBf16>(a, write, st);
    case kKvF16: return launch_move<D, kKvF16>(a, write, st);
    case kKvInt8: return launch_move<D, kKvInt8>(a, write, st);
    default: return launch_move<D, kKvE4m3>(a, write, st);
  }
}

}  // namespace

cudaError_t launch_paged_write(const PagedMoveArgs& a, int head_dim, int fmt, cudaStream_t st) {
  return head_dim == 64 ? launch_move_fmt<64>(a, fmt, true, st) : launch_move_fmt<128>(a, fmt, true, st);
}
cudaError_t launch_paged_read(const PagedMoveArgs& a, int head_dim, int fmt, cudaStream_t st) {
  return head_dim == 64 ? launch_move_fmt<64>(a, fmt, false, st) : launch_move_fmt<128>(a, fmt, false, st);
}

}  // namespace df2
