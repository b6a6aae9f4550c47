// Writing keys and values into the paged cache and reading them back.
//
// Quantised formats: s = max(amax|x| / Q, 2^-126) per (position, KV head) and side, code =
// x / s rounded to nearest even and saturated, value = code * s.  Both divisions are IEEE
// (so a code never depends on how a reciprocal rounds), and |x / s| <= Q up to one rounding.
//
// Both directions are streams over rows of one (token, KV head): 8 channels per lane, the
// keys' and the values' loads issued together, amax by shuffles within the row's lanes, so
// each source element is read once and each code written once.
#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.h"

namespace df2 {
namespace {

constexpr int kThreads = 256;

// Request of packed row t and the row's position in its cache; false if the request's
// range or length is out of bounds (status set) or no request holds the row.
DF2_DEV bool find_position(const PagedReq& q, int t, int& r, int& pos) {
  int lo = 0, hi = q.n_req;  // the last r with begin[r] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(q.begin + mid) <= t) lo = mid;
    else hi = mid;
  }
  const int b0 = __ldg(q.begin + lo), b1 = __ldg(q.begin + lo + 1), len = __ldg(q.kv_len + lo);
  r = lo;
  if (t < b0 || t >= b1) return false;
  if (!paged_request_ok(q, b0, b1, len) || len < b1 - b0) {
    if (q.status) q.status[lo] = 1;  // DFLASH2_E_INVAL
    return false;
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

// Codes of 8 channels; `ok` is false where the row holds an infinity or a NaN (zero codes).
template <int FMT>
DF2_DEV uint2 codes8(const float (&x)[8], float scale, bool ok) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = ok ? __fdiv_rn(x[i], scale) : 0.f;
    uint32_t b;
    if constexpr (FMT == kKvInt8) {
      int c = __float2int_rn(y);
      c = c > 127 ? 127 : (c < -127 ? -127 : c);
      b = static_cast<uint32_t>(c) & 0xFFu;
    } else {
      b = __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
    }
    w[i >> 2] |= b << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

// One row (token, KV head) per D / 8 lanes.
template <int D, int FMT, int T>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ PagedMoveArgs a) {
  constexpr int kLanes = D / 8;
  const long long item = static_cast<long long>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int ch = (threadIdx.x % kLanes) * 8;
  const bool in = item < static_cast<long long>(a.rq.n_tokens) * a.c.n_kv;
  const int t = in ? static_cast<int>(item / a.c.n_kv) : 0, h = in ? static_cast<int>(item % a.c.n_kv) : 0;
  float kx[8], vx[8];
  if (in) {
    load8<T>(a.k.p, t * a.k.token_stride + h * a.k.head_stride + ch, kx);
    load8<T>(a.v.p, t * a.v.token_stride + h * a.v.head_stride + ch, vx);
  }
  int r, pos;
  long long off = 0, soff = 0;
  const bool go = in && find_position(a.rq, t, r, pos) && find_row(a.c, a.rq, r, pos, h, off, soff);
  // a row's lanes decide alike, so the shuffles of the rows that stay need only their own lanes;
  // idle rows take part with zeros to keep the warp together
  if (!go) {
#pragma unroll
    for (int i = 0; i < 8; ++i) kx[i] = vx[i] = 0.f;
  }
  if constexpr (FMT == kKvBf16 || FMT == kKvF16) {
    if (!go) return;
    store8<FMT == kKvBf16 ? kTBf16 : kTF16>(a.c.k, off + ch, kx);
    store8<FMT == kKvBf16 ? kTBf16 : kTF16>(a.c.v, off + ch, vx);
  } else {
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // |x| as bits: ordered as the values are, infinity above every number and NaN above
      // infinity, so a nonfinite element always wins
      mk = max(mk, __float_as_uint(kx[i]) & 0x7FFFFFFFu);
      mv = max(mv, __float_as_uint(vx[i]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    if (!go) return;
    const bool okk = mk < 0x7F800000u, okv = mv < 0x7F800000u;
    constexpr float kQ = FMT == kKvInt8 ? 127.f : 448.f;
    float sk = __fdiv_rn(__uint_as_float(mk), kQ), sv = __fdiv_rn(__uint_as_float(mv), kQ);
    if (okk) sk = fmaxf(sk, 1.17549435e-38f);  // 2^-126
    if (okv) sv = fmaxf(sv, 1.17549435e-38f);
    *reinterpret_cast<uint2*>(a.c.k + off + ch) = codes8<FMT>(kx, sk, okk);
    *reinterpret_cast<uint2*>(a.c.v + off + ch) = codes8<FMT>(vx, sv, okv);
    if (ch == 0) {
      a.c.k_scale[soff] = sk;
      a.c.v_scale[soff] = sv;
    }
  }
}

template <int FMT>
DF2_DEV void read8(const char* pool, const float* scales, long long off, long long soff, int ch, float (&x)[8]) {
  if constexpr (FMT == kKvBf16 || FMT == kKvF16) {
    load8<FMT == kKvBf16 ? kTBf16 : kTF16>(pool, off + ch, x);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(pool + off + ch);
    const float s = scales[soff];
    const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = (ww[i >> 2] >> (8 * (i & 3))) & 0xFFu;
      float c;
      if constexpr (FMT == kKvInt8) {
        c = static_cast<float>(static_cast<int8_t>(b));
      } else {
        const __half_raw hr = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
        c = __half2float(*reinterpret_cast<const __half*>(&hr));
      }
      x[i] = c * s;
    }
  }
}

template <int D, int FMT, int T>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ PagedMoveArgs a) {
  constexpr int kLanes = D / 8;
  const long long item = static_cast<long long>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int ch = (threadIdx.x % kLanes) * 8;
  if (item >= static_cast<long long>(a.rq.n_tokens) * a.c.n_kv) return;
  const int t = static_cast<int>(item / a.c.n_kv), h = static_cast<int>(item % a.c.n_kv);
  int r, pos;
  if (!find_position(a.rq, t, r, pos)) return;
  long long off, soff;
  float kx[8], vx[8];
  if (find_row(a.c, a.rq, r, pos, h, off, soff)) {
    read8<FMT>(a.c.k, a.c.k_scale, off, soff, ch, kx);
    read8<FMT>(a.c.v, a.c.v_scale, off, soff, ch, vx);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) kx[i] = vx[i] = 0.f;
  }
  store8<T>(a.k.p, t * a.k.token_stride + h * a.k.head_stride + ch, kx);
  store8<T>(a.v.p, t * a.v.token_stride + h * a.v.head_stride + ch, vx);
}

template <int D, int FMT>
cudaError_t launch_move(const PagedMoveArgs& a, bool write, cudaStream_t st) {
  const long long items = static_cast<long long>(a.rq.n_tokens) * a.c.n_kv;
  const int per = kThreads / (D / 8);
  const dim3 grid(static_cast<unsigned>((items + per - 1) / per));
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
