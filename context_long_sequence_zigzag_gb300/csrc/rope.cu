// rope.cu — rotary positions of queries and keys, and new tokens into a paged
// cache with their keys turned on the way.
//
// Angles.  A position p times a frequency f, in turns, modulo 1, is all that
// sine and cosine need, and an integer product modulo 2^64 of p and the 64-bit
// fraction f / (2 pi) gives exactly that, for positions near or far, of either
// sign.  The nearest quarter turn is split off in integers; the rest, at most
// an eighth of a turn, goes to sincospif in FP32 (rounded to 24 bits there: off
// by at most 2^-25 of an eighth of a turn).
//
// Both kernels only move memory: a CTA takes a tile of tokens, computes the
// tile's sines and cosines once into shared memory (one a token and pair,
// whatever the number of heads), and each thread then keeps the few that its
// 16 bytes of a head need in registers and streams through the heads.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 256;
// eight 16-byte loads of a thread in flight at 64 registers (a 64K prompt's queries and keys: 217 us; left to 80
// registers 258 us, at five CTAs an SM 283 us, with four loads in flight 248 us)
constexpr int kCtasPerSm = 4;

template <typename E>
struct Vec;  // 16 bytes of a row
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void unpack(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
  __device__ static uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void unpack(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = reinterpret_cast<const uint32_t&>(p);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* p) { *p = __float2bfloat16_rn(x); }

// factor * (cos, sin) of position * turns / 2^64 turns
__device__ __forceinline__ float2 turn_of(uint64_t turns, int32_t position, float factor) {
  const uint64_t t = turns * uint64_t(int64_t(position));
  const uint32_t quarter = uint32_t((t + (uint64_t(1) << 61)) >> 62);
  const int64_t rest = int64_t(t - (uint64_t(quarter) << 62));  // -2^61 .. 2^61
  float s, c;
  sincospif(float(int32_t((rest + (int64_t(1) << 31)) >> 32)) * 0x1p-31f, &s, &c);
  const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
  const float f = quarter & 2 ? -factor : factor;
  return make_float2(f * x, f * y);
}

// Position of a row on the axis of pair i.
__device__ __forceinline__ int32_t position_of(const Rope& r, const int32_t* positions, int64_t row, int32_t stride,
                                               int i, int32_t* err) {
  int32_t axis = r.axis ? __ldg(r.axis + i) : 0;
  if (axis < 0 || axis >= r.axes) {
    kv_error(err, kKvAxis);
    axis = 0;
  }
  return __ldg(positions + row * stride + axis);
}

// One head row after another (in and out advance by their strides), the
// 16-byte pieces that start at channel `ch` (and `ch2`, the partners of HALVES).
// cs: cosines and sines of the piece's pairs.
enum Piece { kCopy, kHalves, kAdjacent };

template <typename E, Piece P, int U>
__device__ __forceinline__ void stream_some(const E* in, int64_t in_stride, E* out, int64_t out_stride, int half,
                                            const float2* cs) {
  constexpr int N = Vec<E>::N;
  uint4 a[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    a[u] = __ldcs(reinterpret_cast<const uint4*>(in + u * in_stride));
    if (P == kHalves) b[u] = __ldcs(reinterpret_cast<const uint4*>(in + u * in_stride + half));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (P == kCopy) {
      __stcs(reinterpret_cast<uint4*>(out + u * out_stride), a[u]);
      continue;
    }
    float x[N], y[N];
    Vec<E>::unpack(a[u], x);
    if (P == kHalves) {
      Vec<E>::unpack(b[u], y);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float p = x[i], q = y[i];
        x[i] = fmaf(p, cs[i].x, -(q * cs[i].y));
        y[i] = fmaf(q, cs[i].x, p * cs[i].y);
      }
      __stcs(reinterpret_cast<uint4*>(out + u * out_stride), Vec<E>::pack(x));
      __stcs(reinterpret_cast<uint4*>(out + u * out_stride + half), Vec<E>::pack(y));
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float p = x[i], q = x[i + 1];
        x[i] = fmaf(p, cs[i / 2].x, -(q * cs[i / 2].y));
        x[i + 1] = fmaf(q, cs[i / 2].x, p * cs[i / 2].y);
      }
      __stcs(reinterpret_cast<uint4*>(out + u * out_stride), Vec<E>::pack(x));
    }
  }
}
template <typename E, Piece P>
__device__ __forceinline__ void stream_heads(const E* in, int64_t in_stride, E* out, int64_t out_stride, int half,
                                             const float2* cs, int heads) {
  int h = 0;
  if constexpr (P != kHalves)  // (one load a head)
    for (; h + 8 <= heads; h += 8, in += 8 * in_stride, out += 8 * out_stride)
      stream_some<E, P, 8>(in, in_stride, out, out_stride, half, cs);
  for (; h + 4 <= heads; h += 4, in += 4 * in_stride, out += 4 * out_stride)
    stream_some<E, P, 4>(in, in_stride, out, out_stride, half, cs);
  for (; h < heads; ++h, in += in_stride, out += out_stride)
    stream_some<E, P, 1>(in, in_stride, out, out_stride, half, cs);
}

// Heads heads of one token, piece p of every row.  cs: the token's.
template <typename E, bool ADJ>
__device__ __forceinline__ void token_piece(const Rope& r, int p, int turned, const E* in, int64_t in_stride, E* out,
                                            int64_t out_stride, int heads, const float2* cs, bool back) {
  constexpr int N = Vec<E>::N, M = ADJ ? N / 2 : N;
  if (p < turned) {
    float2 mine[M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      mine[i] = cs[p * M + i];
      if (back) mine[i].y = -mine[i].y;
    }
    const int ch = r.first + p * N;
    stream_heads<E, ADJ ? kAdjacent : kHalves>(in + ch, in_stride, out + ch, out_stride, r.pairs, mine, heads);
  } else {
    int ch = (p - turned) * N;
    if (r.pairs && ch >= r.first) ch += 2 * r.pairs;
    stream_heads<E, kCopy>(in + ch, in_stride, out + ch, out_stride, 0, nullptr, heads);
  }
}

// The same of one head row, by single channels: for channels that do not come
// in whole 16-byte pieces.  i: a pair, or (from r.pairs on) a channel to copy.
template <typename E>
__device__ __forceinline__ void token_scalar(const Rope& r, int i, const E* in, int64_t in_stride, E* out,
                                             int64_t out_stride, int heads, const float2* cs, bool back) {
  if (i < r.pairs) {
    const float c = cs[i].x, s = back ? -cs[i].y : cs[i].y;
    const int ca = r.adjacent ? r.first + 2 * i : r.first + i, cb = r.adjacent ? ca + 1 : ca + r.pairs;
    for (int h = 0; h < heads; ++h, in += in_stride, out += out_stride) {
      const float a = to_f(in[ca]), b = to_f(in[cb]);
      from_f(fmaf(a, c, -(b * s)), out + ca);
      from_f(fmaf(b, c, a * s), out + cb);
    }
  } else {
    int ch = i - r.pairs;
    if (ch >= r.first) ch += 2 * r.pairs;
    for (int h = 0; h < heads; ++h, in += in_stride, out += out_stride) out[ch] = in[ch];
  }
}

// How a CTA's threads share a tile: `per_row` pieces a head row, a thread each
// as far as the threads go; so many rows at a time, a token's heads in `groups` parts.
struct Split {
  int tile, per_row, turned, groups;
};
// f(piece, token, group) for every one of n tokens
template <typename F>
__device__ __forceinline__ void share(const Split& s, int n, F f) {
  const int across = min(s.per_row, kThreads), rows = kThreads / across;
  const int p0 = threadIdx.x % across, slot = threadIdx.x / across;
  if (slot >= rows) return;
  for (int it = slot; it < n * s.groups; it += rows)
    for (int p = p0; p < s.per_row; p += across) f(p, it / s.groups, it % s.groups);
}

enum Form { kFormHalves, kFormAdjacent, kFormScalar };

template <typename E, Form F>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) rope_kernel(const RopeArgs a, const Split sp) {
  extern __shared__ float2 cs[];  // [tile][pairs]
  const int64_t t0 = int64_t(blockIdx.x) * sp.tile;
  const int n = int(min(int64_t(sp.tile), a.tokens - t0));
  for (int i = threadIdx.x; i < n * a.r.pairs; i += kThreads) {
    const int t = i / a.r.pairs, pr = i - t * a.r.pairs;
    cs[i] = turn_of(__ldg(a.r.turns + pr), position_of(a.r, a.positions, t0 + t, a.pos_stride, pr, a.err), a.r.factor);
  }
  __syncthreads();
  const int all = a.heads[0] + a.heads[1];
  share(sp, n, [&](int p, int t, int g) {
    const int h0 = all * g / sp.groups, h1 = all * (g + 1) / sp.groups;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int base = x ? a.heads[0] : 0;
      const int lo = max(h0, base) - base, hi = min(h1, base + a.heads[x]) - base;
      if (lo >= hi || (p >= sp.turned && a.in[x] == a.out[x])) continue;  // (in place, what does not turn stays)
      const int64_t at = ((t0 + t) * a.heads[x] + lo) * a.d;
      const E* in = static_cast<const E*>(a.in[x]) + at;
      E* out = static_cast<E*>(a.out[x]) + at;
      if constexpr (F == kFormScalar)
        token_scalar<E>(a.r, p, in, a.d, out, a.d, hi - lo, cs + t * a.r.pairs, a.inverse);
      else
        token_piece<E, F == kFormAdjacent>(a.r, p, sp.turned, in, a.d, out, a.d, hi - lo, cs + t * a.r.pairs, a.inverse);
    }
  });
}

// Sequence b with cu[b] <= t < cu[b + 1], or -1 past the last.
__device__ __forceinline__ int seq_of(const int32_t* cu, int n, int64_t t) {
  if (t >= __ldg(cu + n)) return -1;
  int lo = 0, hi = n - 1;  // the last b with cu[b] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

constexpr int kMostTile = 16;

template <typename E, Form F>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv_append_kernel(const KvAppendArgs a, const Split sp, const Split sv) {
  extern __shared__ float2 cs[];  // [tile][pairs]
  __shared__ int64_t to[kMostTile];   // row of the token's first head in the pool, -1: left out
  __shared__ int32_t row[kMostTile], slot_of[kMostTile];
  const int64_t t0 = int64_t(blockIdx.x) * sp.tile;
  const int n = int(min(int64_t(sp.tile), a.tokens - t0));
  if (threadIdx.x < n) {
    const int t = threadIdx.x;
    int64_t dst = -1, slot = 0;
    int32_t r = 0;
    const int b = seq_of(a.cu, a.c.num_seqs, t0 + t);
    if (b >= 0) {
      slot = int64_t(__ldg(a.start + b)) + (t0 + t - __ldg(a.cu + b));
      r = a.rows ? __ldg(a.rows + t0 + t) : int32_t(t0 + t);
      if (slot < 0 || slot >> a.c.page_shift >= a.c.max_pages) kv_error(a.c.err, kKvSlot);
      else if (r < 0 || r >= a.src_rows) kv_error(a.c.err, kKvRow);
      else {
        const int32_t pg = kv_page(__ldg(a.c.table + int64_t(b) * a.c.max_pages + (slot >> a.c.page_shift)),
                                   a.c.num_pages, a.c.err);
        if (pg >= 0) dst = ((int64_t(pg) * a.c.hkv) << a.c.page_shift) + (slot & ((1 << a.c.page_shift) - 1));
      }
    }
    to[t] = dst, row[t] = r, slot_of[t] = int32_t(slot);
  }
  __syncthreads();
  const int hkv = a.c.hkv;
  auto each = [&](const Split& s, auto f) {
    share(s, n, [&](int p, int t, int g) {
      const int h0 = hkv * g / s.groups, h1 = hkv * (g + 1) / s.groups;
      if (to[t] >= 0 && h0 < h1) f(p, t, h0, h1 - h0);
    });
  };
  // values first: nothing of theirs waits for the angles (a 64K prompt: 89 us; behind the keys 92 us)
  each(sv, [&](int p, int t, int h0, int heads) {
    const int ch = p * Vec<E>::N;
    stream_heads<E, kCopy>(static_cast<const E*>(a.v) + (int64_t(row[t]) * hkv + h0) * a.d_v + ch, a.d_v,
                           static_cast<E*>(a.c.v) + (to[t] + (int64_t(h0) << a.c.page_shift)) * a.d_v + ch,
                           int64_t(a.d_v) << a.c.page_shift, 0, nullptr, heads);
  });
  for (int i = threadIdx.x; i < n * a.r.pairs; i += kThreads) {
    const int t = i / a.r.pairs, pr = i - t * a.r.pairs;
    if (to[t] < 0) continue;
    const int32_t pos =
        a.positions ? position_of(a.r, a.positions, row[t], a.pos_stride, pr, a.c.err) : slot_of[t];
    cs[i] = turn_of(__ldg(a.r.turns + pr), pos, a.r.factor);
  }
  __syncthreads();
  each(sp, [&](int p, int t, int h0, int heads) {
    const E* in = static_cast<const E*>(a.k) + (int64_t(row[t]) * hkv + h0) * a.d_qk;
    E* out = static_cast<E*>(a.c.k) + (to[t] + (int64_t(h0) << a.c.page_shift)) * a.d_qk;
    const int64_t stride = int64_t(a.d_qk) << a.c.page_shift;
    if constexpr (F == kFormScalar)
      token_scalar<E>(a.r, p, in, a.d_qk, out, stride, heads, cs + t * a.r.pairs, false);
    else
      token_piece<E, F == kFormAdjacent>(a.r, p, sp.turned, in, a.d_qk, out, stride, heads, cs + t * a.r.pairs, false);
  });
}

// Tokens of a tile: several where that leaves four waves of CTAs (20011 tokens in fp32: 66 us, with one wave 71 us).
int tile_of(int64_t tokens, int most) {
  return int(std::clamp<int64_t>(tokens / (4 * kCtasPerSm * sm_count()), 1, most));
}

Split split_of(int tile, int per_row, int turned, int heads) {
  const int rows = std::max(kThreads / per_row, 1);
  return {tile, per_row, turned, std::clamp((rows + tile - 1) / tile, 1, std::max(heads, 1))};
}

// Whole 16-byte pieces where the turned channels (both halves of them) start and end at one.
Form form_of(const Rope& r, int n) {
  if (r.pairs == 0) return kFormHalves;
  if (r.first % n) return kFormScalar;
  if (r.adjacent) return 2 * r.pairs % n ? kFormScalar : kFormAdjacent;
  return r.pairs % n ? kFormScalar : kFormHalves;
}

// Threads a head row: of the pieces that turn (`turned`), and with `copies` of the others.
int per_row_of(const Rope& r, Form f, int n, int d, bool copies, int* turned) {
  if (f == kFormScalar) {
    *turned = r.pairs;
    return r.pairs + (copies ? d - 2 * r.pairs : 0);
  }
  *turned = f == kFormAdjacent ? 2 * r.pairs / n : r.pairs / n;
  return *turned + (copies ? (d - 2 * r.pairs) / n : 0);
}

template <typename E, typename G>
void with_form(Form f, G g) {
  switch (f) {
    case kFormHalves: g(std::integral_constant<Form, kFormHalves>{}); break;
    case kFormAdjacent: g(std::integral_constant<Form, kFormAdjacent>{}); break;
    default: g(std::integral_constant<Form, kFormScalar>{});
  }
}

template <typename E>
void rope_typed(const RopeArgs& a, cudaStream_t st) {
  const Form f = form_of(a.r, Vec<E>::N);
  const bool copies = (a.heads[0] && a.in[0] != a.out[0]) || (a.heads[1] && a.in[1] != a.out[1]);
  int turned = 0;
  const int per_row = per_row_of(a.r, f, Vec<E>::N, a.d, copies, &turned);
  const int tile = tile_of(a.tokens, std::max(1, 1024 / a.r.pairs));
  const Split sp = split_of(tile, per_row, turned, a.heads[0] + a.heads[1]);
  const unsigned grid = unsigned((a.tokens + tile - 1) / tile);
  with_form<E>(f, [&](auto form) {
    rope_kernel<E, decltype(form)::value><<<grid, kThreads, size_t(tile) * a.r.pairs * sizeof(float2), st>>>(a, sp);
  });
}

template <typename E>
void append_typed(const KvAppendArgs& a, cudaStream_t st) {
  const Form f = form_of(a.r, Vec<E>::N);
  int turned = 0;
  const int per_row = per_row_of(a.r, f, Vec<E>::N, a.d_qk, true, &turned);
  const int tile = tile_of(a.tokens, kMostTile);
  const Split sp = split_of(tile, per_row, turned, a.c.hkv), sv = split_of(tile, a.d_v / Vec<E>::N, 0, a.c.hkv);
  const unsigned grid = unsigned((a.tokens + tile - 1) / tile);
  with_form<E>(f, [&](auto form) {
    kv_append_kernel<E, decltype(form)::value>
        <<<grid, kThreads, size_t(tile) * a.r.pairs * sizeof(float2), st>>>(a, sp, sv);
  });
}

}  // namespace

int sm_count() {
  static std::atomic<int> counts[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  n = counts[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
    counts[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t st) {
  if (dtype == CP_DT_BF16) rope_typed<__nv_bfloat16>(a, st);
  else rope_typed<float>(a, st);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const KvAppendArgs& a, int dtype, cudaStream_t st) {
  if (dtype == CP_DT_BF16) append_typed<__nv_bfloat16>(a, st);
  else append_typed<float>(a, st);
  return cudaGetLastError();
}

}  // namespace cpattn
