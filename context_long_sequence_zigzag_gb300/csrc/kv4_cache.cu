// kv4_cache.cu — the kernels that write, read back and evict from the 4-bit
// key/value cache (format: include/cp_attn.h; attention over it: kv4_attn.cu).
//
// All three move bytes.  In append and read a thread handles 16 channels, two
// 32-bit words of codes: a token's head of 128 channels is 8 lanes, its
// 64-channel groups are aligned runs of 4, and both the tensor side (32 or 64
// bytes a lane) and the cache side (whole 64-byte rows) are contiguous across
// a warp.  (With one word a thread, the places, addresses and reductions took
// as many instructions as the quantising.)
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "kv4.cuh"
#include "kv4_words.h"
#include "sm103_ptx.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = kKv4Threads;

// 16 channels as they lie in memory
template <typename E>
struct Raw {
  static constexpr int N = int(sizeof(E));
  uint4 u[N];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint32_t word(int i) const {  // i is a constant
    return i % 4 == 0 ? u[i / 4].x : (i % 4 == 1 ? u[i / 4].y : (i % 4 == 2 ? u[i / 4].z : u[i / 4].w));
  }
  // channels 8 w .. 8 w + 7
  __device__ __forceinline__ void half(int w, float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (sizeof(E) == 4)
        x[j] = __uint_as_float(word(8 * w + j));
      else
        x[j] = __uint_as_float(j % 2 ? word(4 * w + j / 2) & 0xffff0000u : word(4 * w + j / 2) << 16);
    }
  }
  // Minimum and maximum over 4 lanes' 16 channels each; NaN where one is NaN
  __device__ __forceinline__ void range(uint32_t lanes, float& lo, float& hi) const {
    if constexpr (sizeof(E) == 4) {
      lo = hi = __uint_as_float(word(0));
#pragma unroll
      for (int j = 1; j < 16; ++j) {
        asm("min.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(__uint_as_float(word(j))));
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(__uint_as_float(word(j))));
      }
#pragma unroll
      for (int s = 1; s < 4; s <<= 1) {
        const float l = __shfl_xor_sync(lanes, lo, s), h = __shfl_xor_sync(lanes, hi, s);
        asm("min.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(l));
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(h));
      }
    } else {  // pairs of bf16, and across the lanes the minimum beside the negated maximum
      uint32_t l = word(0), h = l;
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(l) : "r"(word(j)));
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(h) : "r"(word(j)));
      }
      h ^= 0x80008000u;
      const uint32_t other = __byte_perm(l, h, 0x7632);
      l = __byte_perm(l, h, 0x5410);
      asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(l) : "r"(other));
#pragma unroll
      for (int s = 1; s < 4; s <<= 1) {
        const uint32_t o = __shfl_xor_sync(lanes, l, s);
        asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(l) : "r"(o));
      }
      lo = __uint_as_float(l << 16);
      hi = -__uint_as_float(l & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// The code of x where (x - low) or 1 / s leaves fp32's normal range.
__device__ __noinline__ float far_code(float x, float low, float s) {
  const float d = x - low;
  const float q = isinf(d) ? __fdiv_rn(0.5f * x - 0.5f * low, 0.5f * s) : __fdiv_rn(d, s);
  return fminf(fmaxf(rintf(q), 0.f), 15.f);
}

// Codes of 8 channels, channel j in bits 4j: the integers nearest to (x - low)
// / s, halves to even, of the exact quotient.  (x - low) times an approximate
// 1 / s gives n; what it leaves, r = (x - low) - n s, is exact (n s has 12
// bits, and r is below s), so |r| < s / 2 proves n.  Otherwise n is a step off
// or halfway, which happens (bf16 values over a bf16 scale: one in some
// hundreds); there the rounding error e of x - low and n's last bit decide.
// Channels j and j + 4 go in pairs; four codes are put together as a number in
// base 16.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float low, float s, bool plain) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's last bits are the integer
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const uint64_t inv2 = ptx::f32x2(inv, inv), low2 = ptx::f32x2(-low, -low), magic2 = ptx::f32x2(kMagic, kMagic);
  const uint64_t back2 = ptx::f32x2(-kMagic, -kMagic), minus2 = ptx::f32x2(-s, -s), base2 = ptx::f32x2(16.f, 16.f);
  const float half = 0.5f * s;
  float n[8], r[8], most = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t d = ptx::add_f32x2(ptx::f32x2(x[j], x[j + 4]), low2);
    const uint64_t k = ptx::add_f32x2(ptx::fma_f32x2(d, inv2, magic2), back2);
    ptx::f32x2_split(k, n[j], n[j + 4]);
    ptx::f32x2_split(ptx::fma_f32x2(k, minus2, d), r[j], r[j + 4]);
    most = fmaxf(most, fmaxf(fabsf(r[j]), fabsf(r[j + 4])));
  }
  if (!plain) {
#pragma unroll  // (an index that is not a constant would put x into local memory)
    for (int j = 0; j < 8; ++j) n[j] = far_code(x[j], low, s);
  } else if (most >= half) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(r[j]), step = copysignf(1.f, r[j]);
      if (a >= half) {
        const float d = x[j] - low, b = d - x[j];
        const float e = ((x[j] - (d - b)) + (-low - b)) * step;  // the exact residual's |r| is a + e
        const bool odd = __float_as_uint(n[j] + kMagic) & 1u;
        if (a > half || e > 0.f || (e == 0.f && odd)) n[j] += step;
      }
    }
  }
  uint64_t number = ptx::f32x2(n[3], n[7]);
#pragma unroll
  for (int j = 2; j >= 0; --j) number = ptx::fma_f32x2(number, base2, ptx::f32x2(n[j], n[j + 4]));
  float a, b;
  ptx::f32x2_split(ptx::add_f32x2(number, magic2), a, b);
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
}

// A token's place in the cache and its row outside it.
struct Place {
  uint8_t* sub;  // sub-block of head 0's block (heads are block() bytes apart), or null
  float* weight;  // of head 0 (heads are 64 apart), or null
  int64_t src;
  int32_t row;  // row of the sub-block
};

// Null where token t has no slot (padding, or recorded as an error).
__device__ __forceinline__ Place place_of(const Kv4Cache& c, const Kv4Format& f, const int32_t* cu, const int32_t* start,
                                          const int32_t* rows, int64_t src_rows, int64_t t) {
  Place at{nullptr, nullptr, t, 0};
  const int b = kv4_seq_of(cu, c.num_seqs, t);
  if (b < 0) return at;
  const int64_t slot = int64_t(__ldg(start + b)) + t - __ldg(cu + b);
  if (slot < 0 || slot >= int64_t(c.max_pages) * CP_KV4_PAGE) {
    kv4_error(c, kKv4Slot);
    return at;
  }
  if (rows) at.src = __ldg(rows + t);
  if (at.src < 0 || at.src >= src_rows) {
    kv4_error(c, kKv4Row);
    return at;
  }
  const int page = kv4_page(c, b, int32_t(slot / CP_KV4_PAGE)), row = int32_t(slot % CP_KV4_PAGE);
  if (page < 0) return at;
  at.sub = c.pages + int64_t(page) * c.hkv * f.block() + (row / kKv4Sub) * f.sub();
  if (c.weights) at.weight = c.weights + int64_t(page) * c.hkv * CP_KV4_PAGE + row;
  at.row = row % kKv4Sub;
  return at;
}

constexpr int kAhead = 2;        // pieces a thread of read loads before it writes (64K tokens: 65 us; 1: 75, 3: 73)

// CTAs an SM: as many as leave the registers their place (64K tokens of bf16, 8 heads of 128 + 128: 98 us with 4, 135 with
// 5, whose registers spill; fp32 values take more of them).
template <typename E>
__global__ void __launch_bounds__(kThreads, sizeof(E) == 2 ? 4 : 3) kv4_append_kernel(const Kv4Cache c, const Kv4Format f, const Words n, const E* k,
                                                              const E* v, const float* w, int64_t src_rows,
                                                              const int32_t* rows, const int32_t* cu,
                                                              const int32_t* start, int64_t tokens, int per_block) {
  __shared__ Place places[kKv4MostTokens];
  const int64_t t0 = int64_t(blockIdx.x) * per_block;
  const int here = int(min(int64_t(per_block), tokens - t0));
  if (threadIdx.x < here) places[threadIdx.x] = place_of(c, f, cu, start, rows, src_rows, t0 + threadIdx.x);
  __syncthreads();
  const int all = here * n.words;
  auto load = [&](int i, Raw<E>& x) -> Word {  // the groups of 4 lanes stay whole: all is a multiple of 4
    const Word o = word_of(n, i);
    const Place& at = places[o.token];
    if (at.sub) {
      const E* p = o.is_v ? v + (at.src * c.hkv * n.nv + o.r) * 16 : k + (at.src * n.all_k + o.r) * 16;
      x.load(p);
    } else {
      x.zero();
    }
    return o;
  };
  Raw<E> next;
  Word o_next{};
  if (threadIdx.x < all) o_next = load(threadIdx.x, next);
  for (int i = threadIdx.x; i < all; i += kThreads) {
    const Raw<E> raw = next;
    const Word o = o_next;
    if (i + kThreads < all) o_next = load(i + kThreads, next);
    const Place& at = places[o.token];
    float lo, hi;  // of the group: 4 lanes
    raw.range(0xfu << (threadIdx.x & 28), lo, hi);
    if (!at.sub) continue;
    __nv_bfloat16 low = __float2bfloat16_rd(lo);
    const float lowf = __bfloat162float(low);
    // (max - low) / 15; halved first, so that no finite range overflows. A division: the product with 1 / 7.5 falls to the
    // wrong side of four in ten of the quotients that lie halfway between two scales
    __nv_bfloat16 scale = __float2bfloat16_rn(__fdiv_rn(0.5f * hi - 0.5f * lowf, 7.5f));
    const float s = __bfloat162float(scale);
    uint32_t codes[2] = {0, 0};
    if (!isfinite(lowf) || !isfinite(hi)) {
      low = scale = __ushort_as_bfloat16(0x7fff);
    } else if (s > 0.f) {
      const bool plain = s >= 1.2e-38f && hi - lowf < INFINITY;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float x[8];
        raw.half(w, x);
        codes[w] = codes_of(x, lowf, s, plain);
      }
    }
    uint8_t* sub = at.sub + int64_t(o.head) * f.block();
    const int w0 = 2 * o.word, group = o.word / 4;
    if (o.is_v) {
      uint32_t* to = reinterpret_cast<uint32_t*>(sub + f.vc() + at.row * (f.dv / 2));
      to[f.vword(w0)] = codes[0];
      to[f.vword(w0 + 1)] = codes[1];
      if (o.word % 4 == 0) {
        reinterpret_cast<__nv_bfloat16*>(sub + f.vs())[at.row * f.gv() + group] = scale;
        reinterpret_cast<__nv_bfloat16*>(sub + f.vl())[group * kKv4Sub + at.row] = low;
      }
    } else {
      uint32_t* to = reinterpret_cast<uint32_t*>(sub + f.kc() + at.row * (f.dqk / 2));
      to[f.kword(w0)] = codes[0];
      to[f.kword(w0 + 1)] = codes[1];
      if (o.word % 4 == 0) {
        __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(sub + f.kp()) + at.row * 2 * f.gk() + group;
        p[0] = scale;
        p[f.gk()] = low;
      }
      if (o.word == 0 && at.weight)
        at.weight[int64_t(o.head) * CP_KV4_PAGE] = w ? __ldg(w + int64_t(o.head) * src_rows + at.src) : 0.f;
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4Cache c, const Kv4Format f, const Words n,
                                                            const int32_t* cu, const int32_t* start, int64_t tokens,
                                                            E* k, E* v, int per_block) {
  __shared__ Place places[kKv4MostTokens];
  const int64_t t0 = int64_t(blockIdx.x) * per_block;
  const int here = int(min(int64_t(per_block), tokens - t0));
  if (threadIdx.x < here) places[threadIdx.x] = place_of(c, f, cu, start, nullptr, tokens, t0 + threadIdx.x);
  __syncthreads();
  struct Piece {
    uint32_t codes[2];
    float s, low;
    E* to;  // null: nothing to write
  };
  const int all = here * n.words;
  auto load = [&](int i) {
    Piece x{};
    if (i >= all) return x;
    const Word o = word_of(n, i);
    const Place& at = places[o.token];
    if (!at.sub) return x;
    const uint8_t* sub = at.sub + int64_t(o.head) * f.block();
    const int w0 = 2 * o.word, group = o.word / 4;
    if (o.is_v) {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(sub + f.vc() + at.row * (f.dv / 2));
      x.codes[0] = from[f.vword(w0)];
      x.codes[1] = from[f.vword(w0 + 1)];
      x.s = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(sub + f.vs())[at.row * f.gv() + group]);
      x.low = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(sub + f.vl())[group * kKv4Sub + at.row]);
      x.to = v + (at.src * c.hkv * n.nv + o.r) * 16;
    } else {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(sub + f.kc() + at.row * (f.dqk / 2));
      x.codes[0] = from[f.kword(w0)];
      x.codes[1] = from[f.kword(w0 + 1)];
      const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(sub + f.kp()) + at.row * 2 * f.gk() + group;
      x.s = __bfloat162float(p[0]);
      x.low = __bfloat162float(p[f.gk()]);
      x.to = k + (at.src * n.all_k + o.r) * 16;
    }
    return x;
  };
  for (int i = threadIdx.x; i < all; i += kAhead * kThreads) {
    Piece x[kAhead];  // loads of several in flight
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = load(i + u * kThreads);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (!x[u].to) continue;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)  // (a code in the last bits of 2^23 is 2^23 + n)
          y[j] = fmaf(x[u].s, __uint_as_float(((x[u].codes[w] >> (4 * j)) & 15u) | 0x4b000000u) - 8388608.f, x[u].low);
        store8(x[u].to + 8 * w, y);
      }
    }
  }
}

// ---------------------------------------------------------------- eviction
// Weights as unsigned keys of the same order; NaN above all, -0 = +0.
__device__ __forceinline__ uint32_t rank_key(float x) {
  if (isnan(x)) return 0xffffffffu;
  uint32_t u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;
constexpr int kDigits = 2048;      // bins of an 11-bit digit
constexpr int kSelKeys = 49152;    // keys that a CTA keeps in shared memory
constexpr int kSelParts = 8;        // CTAs of a row at most
constexpr int kSelAhead = 8;        // weights a thread has on their way
constexpr int kSelSlice = 8192;    // slots a CTA takes at least where a row gets several

// Sum of x over the threads before this one; *all gets the sum over all.
// scratch: a word a warp, not used again before the block's next barrier.
template <typename T>
__device__ __forceinline__ T block_before(T x, T* scratch, T* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) scratch[warp] = y;
  __syncthreads();
  T z = scratch[lane];  // kSelThreads / 32 = 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, z, o);
    if (lane >= o) z += u;
  }
  *all = __shfl_sync(0xffffffffu, z, 31);
  const T warps_before = __shfl_sync(0xffffffffu, z, max(warp - 1, 0));
  return y - x + (warp > 0 ? warps_before : 0);
}

// A cluster of CTAs per (sequence, kv head): the slots to keep, in order.
// Each CTA holds the keys of its slice of the row in shared memory (rows too
// long for that are read again).  The key of the last slot that is kept is
// found digit by digit, 11 bits a pass: the CTAs count their slices, and every
// one of them sums the counts over the cluster through distributed shared
// memory.  The slots above the key, and the first `need` of those that equal
// it, then get their places from one scan, a thread having consecutive slots.
// Bound by the latency of its barriers and loads, so: counts of their own for
// each pass, the first taken while the keys are loaded, and the block's
// barrier where a row has one CTA.
__global__ void __launch_bounds__(kSelThreads, 2) kv4_select_kernel(const Kv4Cache c, const int32_t* lengths,
                                                                 int32_t budget, int32_t recent, int32_t* new_lengths,
                                                                 int32_t* kept, int most_keys) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(8) int32_t hist[3][kDigits];
  __shared__ int32_t scratch[3][32], s_digit, s_left;
  __shared__ uint64_t scratch2[32], s_count;
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int parts = int(cluster.num_blocks()), part = int(cluster.block_rank());
  auto sync_row = [&] {
    if (parts == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  ptx::grid_launch_dependents();
  const int64_t row = blockIdx.x / parts;
  const int b = int(row / c.hkv), h = int(row - int64_t(b) * c.hkv);
  const int tid = threadIdx.x;
  const int n = kv4_length(c, lengths, b), keep = min(n, budget);
  int32_t* out = kept + row * budget;
  const int first = part * kSelThreads + tid, step = parts * kSelThreads;
  if (h == 0 && first == 0) new_lengths[b] = keep;
  for (int i = keep + first; i < budget; i += step) out[i] = -1;
  if (n <= budget) {
    for (int i = first; i < n; i += step) out[i] = i;
    return;
  }
  const int m = n - recent;    // slots ranked by weight
  int need = budget - recent;  // of which this many stay (need < m); behind them the recent ones
  for (int i = first; i < recent; i += step) out[need + i] = m + i;
  if (need == 0) return;
  const int slice = (m + parts - 1) / parts, lo = min(part * slice, m), count = min(m, lo + slice) - lo;
  auto weight_key = [&](int j) -> uint32_t {
    const int page = kv4_page(c, b, j / CP_KV4_PAGE);
    return page < 0 ? 0u : rank_key(__ldg(c.weights + (int64_t(page) * c.hkv + h) * CP_KV4_PAGE + j % CP_KV4_PAGE));
  };
  const bool held = count <= most_keys;
  auto key_at = [&](int j) -> uint32_t { return held ? keys[j] : weight_key(lo + j); };
  for (int i = tid; i < 3 * kDigits; i += kSelThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  for (int j0 = tid; j0 < count; j0 += kSelAhead * kSelThreads) {  // all pages, then all weights: two waits
    int32_t page[kSelAhead];
    uint32_t key[kSelAhead];
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kSelAhead; ++u) {
      const int j = j0 + u * kSelThreads;
      page[u] = j < count ? __ldg(c.table + int64_t(b) * c.max_pages + (lo + j) / CP_KV4_PAGE) : 0;
    }
#pragma unroll
    for (int u = 0; u < kSelAhead; ++u) {
      const int j = j0 + u * kSelThreads;
      key[u] = 0;
      if (j < count) {
        if (page[u] >= 0 && page[u] < c.num_pages)
          key[u] = rank_key(__ldg(c.weights + (int64_t(page[u]) * c.hkv + h) * CP_KV4_PAGE + (lo + j) % CP_KV4_PAGE));
        else
          bad = true;
      }
    }
    if (bad) kv4_error(c, kKv4Page);
#pragma unroll
    for (int u = 0; u < kSelAhead; ++u) {
      const int j = j0 + u * kSelThreads;
      if (j >= count) break;
      if (held) keys[j] = key[u];
      atomicAdd(&hist[0][key[u] >> 21], 1);
    }
  }
  uint32_t prefix = 0, known = 0;  // known: the bits of it that are found
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    if (pass > 0)
      for (int j = tid; j < count; j += kSelThreads) {
        const uint32_t key = key_at(j);
        if ((key & known) == prefix) atomicAdd(&hist[pass][(key >> shift) & digits], 1);
      }
    sync_row();
    // thread t sums digits 2047 - 2t and 2046 - 2t
    int have[2] = {0, 0};
#pragma unroll
    for (int q = 0; q < kSelParts; ++q) {
      if (q >= parts) break;
      const int2 two = *reinterpret_cast<const int2*>(cluster.map_shared_rank(hist[pass], q) + kDigits - 2 - 2 * tid);
      have[0] += two.y;
      have[1] += two.x;
    }
    int all;
    const int above = block_before(have[0] + have[1], scratch[pass], &all);
    if (above < need && need <= above + have[0] + have[1]) {
      const int low = need > above + have[0];
      s_digit = kDigits - 1 - 2 * tid - low;
      s_left = need - above - (low ? have[0] : 0);
    }
    __syncthreads();
    prefix |= uint32_t(s_digit) << shift;
    known |= digits << shift;
    need = s_left;
  }
  // ---- places: each thread's run of slots (an odd number, so that a warp's reads meet no bank twice)
  const int run = ((count + kSelThreads - 1) / kSelThreads) | 1;
  const int j0 = min(tid * run, count), j1 = min(j0 + run, count);
  uint64_t mine = 0;  // slots above the key, and equal to it in the upper half
  for (int j = j0; j < j1; ++j) {
    const uint32_t key = key_at(j);
    mine += key > prefix ? 1ull : (key == prefix ? 1ull << 32 : 0ull);
  }
  uint64_t all, before = block_before(mine, scratch2, &all);
  if (parts > 1) {
    if (tid == 0) s_count = all;
    cluster.sync();
    for (int q = 0; q < part; ++q) before += *cluster.map_shared_rank(&s_count, q);
    cluster.sync();  // (no CTA leaves while its counts are read)
  }
  int above = int(uint32_t(before)), same = int(before >> 32);
  for (int j = j0; j < j1; ++j) {
    const uint32_t key = key_at(j);
    if (key > prefix) {
      out[above + min(same, need)] = lo + j;
      ++above;
    } else if (key == prefix) {
      if (same < need) out[above + same] = lo + j;
      ++same;
    }
  }
}

// A warp per sub-block of 32 kept slots: codes, parameters and weights move as they are.
__global__ void __launch_bounds__(kThreads) kv4_move_kernel(const Kv4Cache c, const Kv4Cache to, const Kv4Format f,
                                                            int32_t budget, const int32_t* new_lengths,
                                                            const int32_t* kept) {
  const int lane = threadIdx.x & 31;
  const int subs = (budget + kKv4Sub - 1) / kKv4Sub;
  const int64_t unit = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  ptx::grid_wait_previous();  // launched while the selection runs
  if (unit >= int64_t(subs) * c.num_seqs * c.hkv) return;
  const int64_t bh = unit / subs;
  const int u = int(unit - bh * subs), b = int(bh / c.hkv), h = int(bh - int64_t(b) * c.hkv);
  // plain loads of what the selection writes: __ldg is only for data that nothing writes while the kernel lives
  const int n = min(new_lengths[b], budget), first = u * kKv4Sub;
  if (first >= n) return;
  const int dst_page = kv4_page(to, b, first / CP_KV4_PAGE);
  if (dst_page < 0) return;
  const int64_t dst_block = int64_t(dst_page) * c.hkv + h;
  uint8_t* dst = to.pages + dst_block * f.block() + (first % CP_KV4_PAGE) / kKv4Sub * f.sub();
  // where this lane's slot comes from: sub-block (or null) and row
  const uint8_t* src = nullptr;
  int row = 0;
  if (first + lane < n) {
    const int j = kept[bh * budget + first + lane];
    const bool held = j >= 0 && j < c.max_pages * CP_KV4_PAGE;  // (a slot of the table)
    if (!held) kv4_error(c, kKv4Slot);
    const int page = held ? kv4_page(c, b, j / CP_KV4_PAGE) : -1;
    if (page >= 0) {
      const int64_t block = int64_t(page) * c.hkv + h;
      src = c.pages + block * f.block() + (j % CP_KV4_PAGE) / kKv4Sub * f.sub();
      row = j % kKv4Sub;
      to.weights[dst_block * CP_KV4_PAGE + first % CP_KV4_PAGE + lane] =
          c.weights ? __ldg(c.weights + block * CP_KV4_PAGE + j % CP_KV4_PAGE) : 0.f;
    }
  }
  const uint64_t src_bits = reinterpret_cast<uint64_t>(src);
  auto from = [&](int t, int* r) {
    *r = __shfl_sync(0xffffffffu, row, t);
    return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, src_bits, t));
  };
  // rows of `bytes` (a multiple of sizeof(T)) at offset off, token t's being at t * bytes
  auto move_rows = [&](int off, int bytes, auto unit_) {
    using T = decltype(unit_);
    const int per = bytes / int(sizeof(T));
    constexpr int kAtOnce = 4;
    for (int i0 = 0; i0 < kKv4Sub * per; i0 += 32 * kAtOnce) {  // kKv4Sub * per is a multiple of 32: the warp stays whole
      T x[kAtOnce];
      bool have[kAtOnce] = {};
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (i0 + 32 * u >= kKv4Sub * per) break;
        const int i = i0 + 32 * u + lane, t = i / per, e = i - t * per;
        int r;
        const uint8_t* s = from(t, &r);
        have[u] = s != nullptr;
        if (have[u]) x[u] = __ldg(reinterpret_cast<const T*>(s + off) + r * per + e);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (have[u]) reinterpret_cast<T*>(dst + off)[i0 + 32 * u + lane] = x[u];
    }
  };
  move_rows(f.kc(), f.dqk / 2, uint4{});
  move_rows(f.vc(), f.dv / 2, uint4{});
  move_rows(f.kp(), f.gk() * 4, uint32_t{});
  move_rows(f.vs(), f.gv() * 2, uint16_t{});
  if (src)
    for (int g = 0; g < f.gv(); ++g)
      reinterpret_cast<uint16_t*>(dst + f.vl())[g * kKv4Sub + lane] =
          __ldg(reinterpret_cast<const uint16_t*>(src + f.vl()) + g * kKv4Sub + row);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Cache& c, int dqk, int dv, int dtype, const void* k, const void* v,
                              const float* w, int64_t src_rows, const int32_t* rows, const int32_t* cu,
                              const int32_t* start, int64_t tokens, cudaStream_t st) {
  const Words n = words_of(c.hkv, dqk, dv);
  const int per = kv4_tokens_per_block(n.words, tokens, kv4_sm_count());
  const unsigned grid = unsigned((tokens + per - 1) / per);
  if (dtype == CP_DT_BF16)
    kv4_append_kernel<<<grid, kThreads, 0, st>>>(c, Kv4Format(dqk, dv), n, static_cast<const __nv_bfloat16*>(k),
                                                 static_cast<const __nv_bfloat16*>(v), w, src_rows, rows, cu, start,
                                                 tokens, per);
  else
    kv4_append_kernel<<<grid, kThreads, 0, st>>>(c, Kv4Format(dqk, dv), n, static_cast<const float*>(k),
                                                 static_cast<const float*>(v), w, src_rows, rows, cu, start, tokens,
                                                 per);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Cache& c, int dqk, int dv, int dtype, const int32_t* cu, const int32_t* start,
                            int64_t tokens, void* k, void* v, cudaStream_t st) {
  const Words n = words_of(c.hkv, dqk, dv);
  const int per = kv4_tokens_per_block(n.words, tokens, kv4_sm_count());
  const unsigned grid = unsigned((tokens + per - 1) / per);
  if (dtype == CP_DT_BF16)
    kv4_read_kernel<<<grid, kThreads, 0, st>>>(c, Kv4Format(dqk, dv), n, cu, start, tokens,
                                               static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), per);
  else
    kv4_read_kernel<<<grid, kThreads, 0, st>>>(c, Kv4Format(dqk, dv), n, cu, start, tokens, static_cast<float*>(k),
                                               static_cast<float*>(v), per);
  return cudaGetLastError();
}

cudaError_t launch_kv4_evict(const Kv4Cache& c, int dqk, int dv, const int32_t* lengths, int32_t budget,
                             int32_t recent, const Kv4Cache& to, int32_t* new_lengths, int32_t* kept,
                             cudaStream_t st) {
  // CTAs a row by the longest sequence that the table can hold
  const int64_t most = int64_t(c.max_pages) * CP_KV4_PAGE;
  int parts = 1;
  while (parts < kSelParts && int64_t(parts) * kSelSlice < most) parts *= 2;
  const int keys = int(std::min<int64_t>(kSelKeys, (most + parts - 1) / parts));
  static std::atomic<uint64_t> ready{0};  // devices whose kernel may use that much shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kv4_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  cudaLaunchAttribute shape{};
  shape.id = cudaLaunchAttributeClusterDimension;
  shape.val.clusterDim.x = unsigned(parts);
  shape.val.clusterDim.y = shape.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(c.num_seqs) * unsigned(c.hkv) * unsigned(parts));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = size_t(keys) * 4;
  cfg.stream = st;
  cfg.attrs = &shape;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_select_kernel, c, lengths, budget, recent, new_lengths, kept, keys);
  if (e != cudaSuccess) return e;
  const int64_t units = int64_t((budget + kKv4Sub - 1) / kKv4Sub) * c.num_seqs * c.hkv;
  const int64_t grid = (units + kThreads / 32 - 1) / (kThreads / 32);
  shape.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  shape.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv4_move_kernel, c, to, Kv4Format(dqk, dv), budget, static_cast<const int32_t*>(new_lengths),
                            static_cast<const int32_t*>(kept));
}

}  // namespace cpattn
