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
#include "paged_move.cuh"

namespace df2 {
namespace {

constexpr int kThreads = kMoveThreads;

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
        put8<D, FMT, T>(a.c, side, o, so, ch, in, x[i][side]);
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
