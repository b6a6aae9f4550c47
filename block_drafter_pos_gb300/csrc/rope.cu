// Rotary positions: rows turned by their tokens' positions, and keys turned on their way into the paged cache.
//
// Pair i of a head is turned by p f_i.  The plan holds f_i / (2 pi) as a fraction of 2^64 of a turn, so p times it
// modulo 2^64 is the angle with whole turns gone: exact for every position, by one 64-bit multiplication and without a
// range reduction.  As a signed number it is a half turn either way, which rounds once to fp32 for sincospif; products
// and sums are fp32, each output rounded once.
//
// Both kernels are streams: a token's cosines and sines are computed once into shared memory and serve all its heads,
// and an item is 16 channels of a head (8 pairs), two 16-byte loads and stores of 16-bit types.  The table is in
// quarters of an item, so that neighbouring items' 16-byte reads are neighbours too.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "paged_move.cuh"
#include "rope.h"

namespace df2 {
namespace {

constexpr int kThreads = kMoveThreads;

// Cosine and sine (times the amplitude, and the sign) of pair i at position p.
DF2_DEV float2 turn_of(const RopePlan& plan, int i, int p) {
  const long long t = static_cast<long long>(static_cast<unsigned long long>(static_cast<long long>(p)) * plan.turns[i]);
  float s, c;
  sincospif(static_cast<float>(t) * 0x1p-63f, &s, &c);  // (half turns)
  return make_float2(c * plan.amplitude, s * (plan.amplitude * plan.sign));
}

// A token's table: [4][items] float4, quarter w of item j holds pairs 8 j + 2 w and 8 j + 2 w + 1.
DF2_DEV void put_turn(float4* table, int items, int i, float2 cs) {
  reinterpret_cast<float2*>(table)[((i >> 1 & 3) * items + (i >> 3)) * 2 + (i & 1)] = cs;
}

// Pairs (a, b) turned.
DF2_DEV void turn2(float& a, float& b, float c, float s) {
  const float x = a * c - b * s, y = b * c + a * s;
  a = x, b = y;
}
// The 8 pairs of an item, (lo[i], hi[i]) or, interleaved, neighbours in lo and then in hi.
template <bool IL>
DF2_DEV void turn_item(float (&lo)[8], float (&hi)[8], const float4* table, int items, int j) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float4 t = table[w * items + j];
    if constexpr (IL) {
      float(&v)[8] = w < 2 ? lo : hi;
      turn2(v[4 * (w & 1)], v[4 * (w & 1) + 1], t.x, t.y);
      turn2(v[4 * (w & 1) + 2], v[4 * (w & 1) + 3], t.z, t.w);
    } else {
      turn2(lo[2 * w], hi[2 * w], t.x, t.y);
      turn2(lo[2 * w + 1], hi[2 * w + 1], t.z, t.w);
    }
  }
}

// One item of a head: 16 turned channels (j < items), or up to 16 of those behind them.
template <int T, bool IL>
struct Item {
  float lo[8], hi[8];
  int first, second;  // channels (second < 0: none)
  DF2_DEV void at(int rot, int dim, int items, int j) {
    if (j < items) {
      first = IL ? 16 * j : 8 * j;
      second = IL ? first + 8 : first + (rot >> 1);
    } else {
      first = rot + 16 * (j - items);
      second = first + 8 < dim ? first + 8 : -1;
    }
  }
  DF2_DEV void load(const char* p, long long row) {
    load8<T>(p, row + first, lo);
    if (second >= 0) load8<T>(p, row + second, hi);
  }
  DF2_DEV void store(char* p, long long row) const {
    store8<T>(p, row + first, lo);
    if (second >= 0) store8<T>(p, row + second, hi);
  }
};

struct Quotient {  // n / d for n and d up to 2^16 (the magic number is off by less than d / 2^32)
  uint32_t magic;
  __host__ explicit Quotient(int d) : magic(static_cast<uint32_t>((0x100000000ull + d - 1) / d)), d(d) {}
  DF2_DEV int of(int n) const { return d == 1 ? n : static_cast<int>(__umulhi(n, magic)); }
  int d;
};

// A CTA turns `per` tokens.  Its items are numbered by token, then x's heads and k's, then along the head.
template <int T, bool IL>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int per, Quotient by_token,
                                                        Quotient by_xhead, Quotient by_khead) {
  extern __shared__ float4 table[];  // [per][4][items]
  const int items = a.plan.rot >> 4, pairs = a.plan.rot >> 1;
  const int t0 = blockIdx.x * per, n = min(per, a.n_tokens - t0);
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int t = i / pairs;
    put_turn(table + t * 4 * items, items, i - t * pairs, turn_of(a.plan, i - t * pairs, __ldg(a.positions + t0 + t)));
  }
  __syncthreads();
  const int x_items = a.x_heads * by_xhead.d;
  struct Place {
    const char* src;
    char* dst;
    long long from, to;
    int t, j;
  };
  auto place = [&](int i, Item<T, IL>& it) {
    Place p;
    p.t = by_token.of(i);
    int o = i - p.t * by_token.d;
    const bool x = o < x_items;
    if (!x) o -= x_items;
    const int h = x ? by_xhead.of(o) : by_khead.of(o);
    p.j = o - h * (x ? by_xhead.d : by_khead.d);
    const PagedRows &s = x ? a.x : a.k, &d = x ? a.y : a.ky;
    p.src = s.p, p.dst = d.p;
    p.from = (t0 + p.t) * s.token_stride + h * s.head_stride;
    p.to = (t0 + p.t) * d.token_stride + h * d.head_stride;
    it.at(a.plan.rot, a.dim, items, p.j);
    return p;
  };
  const int total = n * by_token.d;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < total; i += 2 * kThreads * gridDim.y) {
    Item<T, IL> u[2];
    Place p[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int ie = i + e * kThreads * static_cast<int>(gridDim.y);
      p[e].t = -1;
      if (ie < total) {
        p[e] = place(ie, u[e]);
        u[e].load(p[e].src, p[e].from);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (p[e].t < 0) continue;
      if (p[e].j < items) turn_item<IL>(u[e].lo, u[e].hi, table + p[e].t * 4 * items, items, p[e].j);
      u[e].store(p[e].dst, p[e].to);
    }
  }
}

template <int T>
cudaError_t launch_rows(const RopeArgs& a, int num_sms, cudaStream_t st) {
  const int items = a.plan.rot >> 4, rest = (a.dim - a.plan.rot + 15) >> 4;
  const Quotient xh(items + (a.x_copy ? rest : 0)), kh(items + (a.k_copy ? rest : 0));
  const int token = a.x_heads * xh.d + a.k_heads * kh.d;
  // about 8 items a thread while that leaves two CTAs an SM; below, a token a CTA, its items split over up to 4
  int per = std::max(1, std::min({16, 8 * kThreads / token, a.n_tokens / (2 * num_sms)}));
  const int ctas = (a.n_tokens + per - 1) / per;
  const int split = ctas >= num_sms ? 1 : std::max(1, std::min(4, (token + 2 * kThreads - 1) / (2 * kThreads)));
  const size_t smem = static_cast<size_t>(per) * 4 * items * sizeof(float4);
  const Quotient tok(token);
  if (a.plan.interleaved) rope_kernel<T, true><<<dim3(ctas, split), kThreads, smem, st>>>(a, per, tok, xh, kh);
  else rope_kernel<T, false><<<dim3(ctas, split), kThreads, smem, st>>>(a, per, tok, xh, kh);
  return cudaGetLastError();
}

// 8 tokens a CTA.  blockIdx.y = 0: their keys and values, a warp per token, as dflash2_paged_write stores them; the
// others: a share of the query heads each.
template <int D, int FMT, int T>
__global__ void __launch_bounds__(kThreads) rope_write_kernel(const __grid_constant__ RopeWriteArgs a) {
  constexpr int kTokens = kThreads / 32, kLanes = D / 8, kMaxItems = D / 16;
  __shared__ float4 table[kTokens][4 * kMaxItems];
  __shared__ int good[kTokens];
  const PagedMoveArgs& m = a.move;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x * kTokens + wid;
  const int rot = a.plan.rot, items = rot >> 4, half = rot >> 1;
  if (blockIdx.y == 0) flag_requests(m.rq);
  int r = 0, pos = 0;
  const bool found = t < m.rq.n_tokens && find_position(m.rq, t, r, pos);
  if (found) {
    const int p = a.positions ? __ldg(a.positions + t) : pos;
    for (int i = lane; i < half; i += 32) put_turn(table[wid], items, i, turn_of(a.plan, i, p));
  }
  if (lane == 0) good[wid] = found;
  if (blockIdx.y > 0) {
    __syncthreads();
    const int per_head = items + (a.q_copy ? (D - rot + 15) >> 4 : 0);
    const int h0 = static_cast<int>(static_cast<long long>(a.q_heads) * (blockIdx.y - 1) / (gridDim.y - 1));
    const int h1 = static_cast<int>(static_cast<long long>(a.q_heads) * blockIdx.y / (gridDim.y - 1));
    const int per_token = (h1 - h0) * per_head;
    auto turn = [&](auto il) {
      constexpr bool IL = decltype(il)::value;
      for (int w = 0; w < kTokens; ++w) {
        if (!good[w]) continue;
        const long long row = blockIdx.x * kTokens + w;
        for (int i = threadIdx.x; i < per_token; i += kThreads) {
          const int h = i / per_head, j = i - h * per_head;
          Item<T, IL> u;
          u.at(rot, D, items, j);
          u.load(a.q.p, row * a.q.token_stride + (h0 + h) * a.q.head_stride);
          if (j < items) turn_item<IL>(u.lo, u.hi, table[w], items, j);
          u.store(a.y.p, row * a.y.token_stride + (h0 + h) * a.y.head_stride);
        }
      }
    };
    if (a.plan.interleaved) turn(std::true_type{});
    else turn(std::false_type{});
    return;
  }
  __syncwarp();
  if (!found) return;
  long long off, soff;
  if (!find_row(m.c, m.rq, r, pos, 0, off, soff)) return;  // (the whole warp)
  const char* const pk = m.k.p + t * m.k.token_stride * (T == kTF32 ? 4 : 2);
  const char* const pv = m.v.p + t * m.v.token_stride * (T == kTF32 ? 4 : 2);
  const int pieces = m.c.n_kv * kLanes, ch = (lane % kLanes) * 8;
  // this lane's channels' partners and turns, the same in every head
  const bool turned = ch < rot, upper = ch >= half;
  const int partner = upper ? ch - half : ch + half;
  float cs[8], sn[8];
  if (turned) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (a.plan.interleaved) {
        const float4 q = table[wid][(2 * (ch >> 3 & 1) + (w & 1)) * items + (ch >> 4)];
        if (w < 2) cs[2 * w] = q.x, sn[2 * w] = q.y, cs[2 * w + 1] = q.z, sn[2 * w + 1] = q.w;
      } else {
        const float4 q = table[wid][w * items + ((upper ? partner : ch) >> 3)];
        cs[2 * w] = q.x, sn[2 * w] = upper ? q.y : -q.y, cs[2 * w + 1] = q.z, sn[2 * w + 1] = upper ? q.w : -q.w;
      }
    }
  }
  for (int p0 = 0; p0 < pieces; p0 += 64) {
    float x[2][2][8], b[2][8];
    int h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = p0 + 32 * i + lane;
      h[i] = p < pieces ? p / kLanes : 0;  // (idle lanes redo head 0 and store nothing)
      load8<T>(pk, h[i] * m.k.head_stride + ch, x[i][0]);
      if (turned && !a.plan.interleaved) load8<T>(pk, h[i] * m.k.head_stride + partner, b[i]);
      load8<T>(pv, h[i] * m.v.head_stride + ch, x[i][1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = p0 + 32 * i + lane < pieces;
      const long long o = off + h[i] * m.c.head_stride + ch, so = soff + h[i] * m.c.s_head_stride;
      if (turned) {
        if (a.plan.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) turn2(x[i][0][2 * e], x[i][0][2 * e + 1], cs[e], sn[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][0][e] = x[i][0][e] * cs[e] + b[i][e] * sn[e];
        }
      }
      put8<D, FMT, kTF32>(m.c, 0, o, so, ch, in, x[i][0]);
      put8<D, FMT, T>(m.c, 1, o, so, ch, in, x[i][1]);
    }
  }
}

template <int D, int FMT>
cudaError_t launch_write(const RopeWriteArgs& a, int num_sms, cudaStream_t st) {
  const int ctas = (a.move.rq.n_tokens + kThreads / 32 - 1) / (kThreads / 32);
  // few tokens: their query heads over more CTAs
  const int split = a.q.p ? std::max(1, std::min({8, a.q_heads, 2 * num_sms / ctas})) : 0;
  const dim3 grid(ctas, 1 + split);
  switch (a.move.k.type) {
    case kTBf16: rope_write_kernel<D, FMT, kTBf16><<<grid, kThreads, 0, st>>>(a); break;
    case kTF16: rope_write_kernel<D, FMT, kTF16><<<grid, kThreads, 0, st>>>(a); break;
    default: rope_write_kernel<D, FMT, kTF32><<<grid, kThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_write_fmt(const RopeWriteArgs& a, int fmt, int num_sms, cudaStream_t st) {
  switch (fmt) {
    case kKvBf16: return launch_write<D, kKvBf16>(a, num_sms, st);
    case kKvF16: return launch_write<D, kKvF16>(a, num_sms, st);
    case kKvInt8: return launch_write<D, kKvInt8>(a, num_sms, st);
    default: return launch_write<D, kKvE4m3>(a, num_sms, st);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t st) {
  switch (a.x.type) {
    case kTBf16: return launch_rows<kTBf16>(a, num_sms, st);
    case kTF16: return launch_rows<kTF16>(a, num_sms, st);
    default: return launch_rows<kTF32>(a, num_sms, st);
  }
}

cudaError_t launch_rope_write(const RopeWriteArgs& a, int head_dim, int fmt, int num_sms, cudaStream_t st) {
  return head_dim == 64 ? launch_write_fmt<64>(a, fmt, num_sms, st) : launch_write_fmt<128>(a, fmt, num_sms, st);
}

}  // namespace df2
