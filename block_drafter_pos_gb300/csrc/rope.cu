// Rotary positions: rows turned by their tokens' positions, and keys turned on their way into the paged cache.
//
// Pair i of a head is turned by p f_i.  The plan holds f_i / (2 pi) as a fraction of 2^64 of a turn, so p times it
// modulo 2^64 is the angle with whole turns gone: exact for every position, by one 64-bit multiplication and without a
// range reduction.  As a signed number it is a half turn either way, which rounds once to fp32 for sincospif; products
// and sums are fp32, each output rounded once.
//
// Both kernels are streams: a token's cosines and sines are computed once into shared memory and serve all its heads,
// and an item is 16 channels of a head (8 pairs), two 16-byte loads and stores of 16-bit types.  The table is in
// quarters of an item, so that neighbouring items' 16-byte reads are neighbours too.  A thread has the same item of four tokens
// (of fp32, two) in flight: 32768 tokens of 32 + 8 bf16 heads of 128 (671 MB) 98 us, 6.8 TB/s, the rate of a copy; an item at a time 116.
// 9001 tokens of 28 fp32 heads of 64, 16 channels turned (129 MB): 23 us, 5.6 TB/s.
//
// Into the cache: 30,005 tokens, 64 of 128 channels turned, bf16 to e4m3 (678 MB) 114 us, 5.9 TB/s; the quantisation's
// instructions (65% of the issue slots) run beside the queries' bytes.  64 single tokens: into bf16 5.2 us, into int8 7.7 (9.9 with cold
// caches), a chain of dependent latencies: the request's bounds, position, page, row.  Under the 64 registers of four CTAs an SM a thread
// spills 20 to 24 bytes from bf16 or fp32 rows to 16-bit caches and 52 to 60 from fp32 to 8-bit ones, else nothing.
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
struct Span {
  int first, second;  // channels (second < 0: none)
  bool turned;
  template <bool IL>
  static DF2_DEV Span of(int rot, int dim, int items, int j) {
    Span s;
    s.turned = j < items;
    if (s.turned) {
      s.first = IL ? 16 * j : 8 * j;
      s.second = IL ? s.first + 8 : s.first + (rot >> 1);
    } else {
      s.first = rot + 16 * (j - items);
      s.second = s.first + 8 < dim ? s.first + 8 : -1;
    }
    return s;
  }
};
// 8 channels as they lie in memory.
template <int T>
struct Raw {
  uint4 w[T == kTF32 ? 2 : 1];
  DF2_DEV void load(const char* p, long long off) {
    const uint4* s = reinterpret_cast<const uint4*>(p + off * (T == kTF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (T == kTF32 ? 2 : 1); ++i) w[i] = s[i];
  }
  DF2_DEV void store(char* p, long long off) const {
    uint4* d = reinterpret_cast<uint4*>(p + off * (T == kTF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (T == kTF32 ? 2 : 1); ++i) d[i] = w[i];
  }
  DF2_DEV void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < (T == kTF32 ? 2 : 1); ++i) {
      const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (T == kTF32) {
          x[4 * i + e] = __uint_as_float(v[e]);
        } else {
          const float2 f = unpack2<T == kTBf16>(v[e]);
          x[2 * e] = f.x, x[2 * e + 1] = f.y;
        }
      }
    }
  }
  DF2_DEV void put(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < (T == kTF32 ? 2 : 1); ++i) {
      if constexpr (T == kTF32)
        w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
      else
        w[i] = make_uint4(pack2<T == kTBf16>(x[0], x[1]), pack2<T == kTBf16>(x[2], x[3]), pack2<T == kTBf16>(x[4], x[5]),
                          pack2<T == kTBf16>(x[6], x[7]));
    }
  }
};

// The item of tokens t, t + 1, ... (`n` of them, at most kTogether<T>; those whose bit in `live` is not set are passed over): their
// loads are in flight together.
template <int T>
constexpr int kTogether = T == kTF32 ? 2 : 4;
template <int T, bool IL>
DF2_DEV void turn_tokens(const PagedRows& x, const PagedRows& y, long long t, int h, const Span& s, int n, uint32_t live,
                         const float4* table, int items, int j) {
  Raw<T> lo[kTogether<T>], hi[kTogether<T>];
  const long long from = t * x.token_stride + h * x.head_stride, to = t * y.token_stride + h * y.head_stride;
#pragma unroll
  for (int e = 0; e < kTogether<T>; ++e)
    if (e < n && (live >> e & 1)) {
      lo[e].load(x.p, from + e * x.token_stride + s.first);
      if (s.second >= 0) hi[e].load(x.p, from + e * x.token_stride + s.second);
    }
#pragma unroll
  for (int e = 0; e < kTogether<T>; ++e)
    if (e < n && (live >> e & 1)) {
      if (s.turned) {
        float a[8], b[8];
        lo[e].get(a);
        hi[e].get(b);
        turn_item<IL>(a, b, table + e * 4 * items, items, j);
        lo[e].put(a);
        hi[e].put(b);
      }
      lo[e].store(y.p, to + e * y.token_stride + s.first);
      if (s.second >= 0) hi[e].store(y.p, to + e * y.token_stride + s.second);
    }
}

// A CTA turns `per` tokens.  A thread takes an item (numbered by x's heads and k's, then along the head) of
// up to four tokens at a time.
template <int T, bool IL>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int per, int x_each, int k_each) {
  extern __shared__ float4 table[];  // [per][4][items]
  const int items = a.plan.rot >> 4, pairs = a.plan.rot >> 1;
  const int t0 = blockIdx.x * per, n = min(per, a.n_tokens - t0);
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int t = i / pairs;
    put_turn(table + t * 4 * items, items, i - t * pairs, turn_of(a.plan, i - t * pairs, __ldg(a.positions + t0 + t)));
  }
  __syncthreads();
  const int x_items = a.x_heads * x_each, token = x_items + a.k_heads * k_each, groups = (n + kTogether<T> - 1) / kTogether<T>;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < token * groups; i += kThreads * gridDim.y) {
    const int g = i / token;
    int o = i - g * token;
    const bool x = o < x_items;
    if (!x) o -= x_items;
    const int each = x ? x_each : k_each, h = o / each, j = o - h * each;
    turn_tokens<T, IL>(x ? a.x : a.k, x ? a.y : a.ky, t0 + g * kTogether<T>, h, Span::of<IL>(a.plan.rot, a.dim, items, j),
                       n - g * kTogether<T>, (1u << kTogether<T>) - 1u, table + g * kTogether<T> * 4 * items, items, j);
  }
}

template <int T>
cudaError_t launch_rows(const RopeArgs& a, int num_sms, cudaStream_t st) {
  const int items = a.plan.rot >> 4, rest = (a.dim - a.plan.rot + 15) >> 4;
  const int x_each = items + (a.x_copy ? rest : 0), k_each = items + (a.k_copy ? rest : 0);
  const int token = a.x_heads * x_each + a.k_heads * k_each;
  // about eight CTAs an SM (9001 tokens of 112 items: with four 27 us, with eight 23), of whole groups of tokens, up to 8 tokens or
  // 16 of few items; a token a CTA where there are few, its items split over up to 4
  const int most = token <= kThreads ? 16 : 8, share = a.n_tokens / (8 * num_sms);
  const int per = share >= most ? most : share >= 4 ? share & ~3 : std::max(1, share);
  const int ctas = (a.n_tokens + per - 1) / per;
  const int split = ctas >= num_sms ? 1 : std::max(1, std::min(4, (token + kThreads - 1) / kThreads));
  const size_t smem = static_cast<size_t>(per) * 4 * items * sizeof(float4);
  if (a.plan.interleaved) rope_kernel<T, true><<<dim3(ctas, split), kThreads, smem, st>>>(a, per, x_each, k_each);
  else rope_kernel<T, false><<<dim3(ctas, split), kThreads, smem, st>>>(a, per, x_each, k_each);
  return cudaGetLastError();
}

// 8 tokens to `parts` CTAs.  The first: their keys and values, a warp per token, as dflash2_paged_write stores them; the
// others: a share of the query heads each.  (The CTAs of a token follow one another, so that those bound by the quantisation's
// instructions run beside those bound by memory.)
template <int D, int FMT, int T>
__global__ void __launch_bounds__(kThreads, 4) rope_write_kernel(const __grid_constant__ RopeWriteArgs a, int parts) {
  constexpr int kTokens = kThreads / 32, kLanes = D / 8, kMaxItems = D / 16;
  __shared__ float4 table[kTokens][4 * kMaxItems];
  __shared__ int good[kTokens];
  const PagedMoveArgs& m = a.move;
  const int block = blockIdx.x / parts, part = blockIdx.x - block * parts;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, t = block * kTokens + wid;
  const int rot = a.plan.rot, items = rot >> 4, half = rot >> 1;
  if (part == 0) flag_requests(m.rq);
  int r = 0, pos = 0;
  const bool found = t < m.rq.n_tokens && find_position(m.rq, t, r, pos);
  if (found) {
    const int p = a.positions ? __ldg(a.positions + t) : pos;
    for (int i = lane; i < half; i += 32) put_turn(table[wid], kMaxItems, i, turn_of(a.plan, i, p));
  }
  if (lane == 0) good[wid] = found;
  if (part > 0) {
    __syncthreads();
    const int per_head = items + (a.q_copy ? (D - rot + 15) >> 4 : 0);
    const int h0 = static_cast<int>(static_cast<long long>(a.q_heads) * (part - 1) / (parts - 1));
    const int h1 = static_cast<int>(static_cast<long long>(a.q_heads) * part / (parts - 1));
    const int per_token = (h1 - h0) * per_head;
    uint32_t live = 0;
#pragma unroll
    for (int w = 0; w < kTokens; ++w) live |= (good[w] ? 1u : 0u) << w;
    auto turn = [&](auto il) {
      constexpr bool IL = decltype(il)::value;
      for (int i = threadIdx.x; i < per_token * (kTokens / kTogether<T>); i += kThreads) {
        const int g = i / per_token, o = i - g * per_token, h = o / per_head, j = o - h * per_head;
        turn_tokens<T, IL>(a.q, a.y, static_cast<long long>(block) * kTokens + g * kTogether<T>, h0 + h, Span::of<IL>(rot, D, items, j),
                           kTogether<T>, live >> (g * kTogether<T>), table[g * kTogether<T>], kMaxItems, j);
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
  // this lane's channels' partners, the same in every head
  const bool turned = ch < rot, upper = ch >= half, il = a.plan.interleaved;
  const int partner = upper ? ch - half : ch + half;
  const float4* const turns = table[wid] + (il ? 2 * (ch >> 3 & 1) * kMaxItems + (ch >> 4) : (upper ? partner : ch) >> 3);
  for (int p0 = 0; p0 < pieces; p0 += 64) {
    Raw<T> k[2], b[2], v[2];
    int h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = p0 + 32 * i + lane;
      h[i] = p < pieces ? p / kLanes : 0;  // (idle lanes redo head 0 and store nothing)
      k[i].load(pk, h[i] * m.k.head_stride + ch);
      if (turned && !il) b[i].load(pk, h[i] * m.k.head_stride + partner);
      v[i].load(pv, h[i] * m.v.head_stride + ch);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = p0 + 32 * i + lane < pieces;
      const long long o = off + h[i] * m.c.head_stride + ch, so = soff + h[i] * m.c.s_head_stride;
      float x[8];
      k[i].get(x);
      if (turned && il) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float4 t4 = turns[w * kMaxItems];
          turn2(x[4 * w], x[4 * w + 1], t4.x, t4.y);
          turn2(x[4 * w + 2], x[4 * w + 3], t4.z, t4.w);
        }
      } else if (turned) {
        float y[8];
        b[i].get(y);
        const float sign = upper ? 1.f : -1.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 t4 = turns[w * kMaxItems];
          x[2 * w] = x[2 * w] * t4.x + y[2 * w] * (sign * t4.y);
          x[2 * w + 1] = x[2 * w + 1] * t4.z + y[2 * w + 1] * (sign * t4.w);
        }
      }
      put8<D, FMT, kTF32>(m.c, 0, o, so, ch, in, x);
      v[i].get(x);
      put8<D, FMT, T>(m.c, 1, o, so, ch, in, x);
    }
  }
}

template <int D, int FMT>
cudaError_t launch_write(const RopeWriteArgs& a, int num_sms, cudaStream_t st) {
  const int ctas = (a.move.rq.n_tokens + kThreads / 32 - 1) / (kThreads / 32);
  // few tokens: their query heads over more CTAs
  const int split = a.q.p ? std::max(1, std::min({8, a.q_heads, 2 * num_sms / ctas})) : 0;
  const int parts = 1 + split;
  const dim3 grid(static_cast<unsigned>(ctas) * parts);
  switch (a.move.k.type) {
    case kTBf16: rope_write_kernel<D, FMT, kTBf16><<<grid, kThreads, 0, st>>>(a, parts); break;
    case kTF16: rope_write_kernel<D, FMT, kTF16><<<grid, kThreads, 0, st>>>(a, parts); break;
    default: rope_write_kernel<D, FMT, kTF32><<<grid, kThreads, 0, st>>>(a, parts); break;
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
