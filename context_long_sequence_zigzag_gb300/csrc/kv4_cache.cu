// kv4_cache.cu — the kernels that write, read back and evict from the 4-bit
// key/value cache (format: include/cp_attn.h; attention over it: kv4_attn.cu).
//
// All three move bytes: a thread handles one 32-bit word of codes (8
// channels), so a token's head of 128 channels is 16 lanes, its 64-channel
// groups are aligned runs of 8 lanes, and both the tensor side (16 or 32
// bytes a lane) and the cache side (whole 64-byte rows) are contiguous
// across a warp.
#include "kv4.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
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

// The integer nearest to (x - low) / s, halves to even, of the exact
// quotient.  The quotient in fp32 is off by a few units of 2^-23: only where
// it falls that close to a half is the exact sign of (x - low) - (f + 1/2) s
// needed (f + 1/2 and s have 13 bits together, so the product inside the FMA
// is exact; e is the rounding error of x - low).
__device__ __forceinline__ float code_of(float x, float low, float s) {
  const float d = x - low;
  float q = __fdiv_rn(d, s);
  if (isinf(d)) q = __fdiv_rn(0.5f * x - 0.5f * low, 0.5f * s);
  const float f = floorf(q);
  if (fabsf(q - f - 0.5f) < 1e-5f && f < 16.f) {
    const float bb = d - x;
    const float e = (x - (d - bb)) + (-low - bb);
    const float t = fmaf(-(f + 0.5f), s, d) + e;
    q = t > 0.f ? f + 1.f : (t < 0.f ? f : rintf(f + 0.5f));
  } else {
    q = rintf(q);
  }
  return fminf(fmaxf(q, 0.f), 15.f);
}

// One token's place in the cache.
struct Place {
  uint8_t* sub;      // sub-block of head 0's block; heads are block() bytes apart
  int32_t page, row;  // row 0 .. 63 of the page
};

// Slot of token t; false where there is none (padding, or recorded as an error).
__device__ __forceinline__ bool find_place(const Kv4Cache& c, const Kv4Format& f, const int32_t* cu,
                                           const int32_t* start, int64_t t, Place* at) {
  const int b = kv4_seq_of(cu, c.num_seqs, t);
  if (b < 0) return false;
  const int64_t slot = int64_t(__ldg(start + b)) + t - __ldg(cu + b);
  if (slot < 0 || slot >= int64_t(c.max_pages) * CP_KV4_PAGE) {
    kv4_error(c, kKv4Slot);
    return false;
  }
  at->page = kv4_page(c, b, int32_t(slot / CP_KV4_PAGE));
  if (at->page < 0) return false;
  at->row = int32_t(slot % CP_KV4_PAGE);
  at->sub = c.pages + int64_t(at->page) * c.hkv * f.block() + (at->row / kKv4Sub) * f.sub();
  return true;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4Cache c, const Kv4Format f, const E* k, const E* v,
                                                              const float* w, int64_t src_rows, const int32_t* rows,
                                                              const int32_t* cu, const int32_t* start, int64_t tokens,
                                                              int per_block) {
  const int nk = f.dqk / 8, nv = f.dv / 8, words = c.hkv * (nk + nv);
  const int64_t t0 = int64_t(blockIdx.x) * per_block;
  const int n = int(min(int64_t(per_block), tokens - t0)) * words;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int64_t t = t0 + i / words;
    int r = i % words;
    Place at;
    if (!find_place(c, f, cu, start, t, &at)) continue;
    const int64_t src = rows ? int64_t(__ldg(rows + t)) : t;
    if (src < 0 || src >= src_rows) {
      kv4_error(c, kKv4Row);
      continue;
    }
    const bool is_v = r >= c.hkv * nk;
    if (is_v) r -= c.hkv * nk;
    const int per = is_v ? nv : nk, head = r / per, word = r % per, group = word / 8;
    float x[8];
    load8(is_v ? v + (src * c.hkv * nv + r) * 8 : k + (src * c.hkv * nk + r) * 8, x);
    // the group's minimum and maximum over its 8 lanes; x - x is NaN for NaN and infinities
    float lo = x[0], hi = x[0], bad = x[0] - x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) lo = fminf(lo, x[j]), hi = fmaxf(hi, x[j]), bad += x[j] - x[j];
    const uint32_t lanes = 0xffu << (threadIdx.x & 24);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(lanes, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(lanes, hi, o));
      bad += __shfl_xor_sync(lanes, bad, o);
    }
    __nv_bfloat16 low = __float2bfloat16_rd(lo);
    const float lowf = __bfloat162float(low);
    // (max - low) / 15; halved first, so that no finite range overflows
    __nv_bfloat16 scale = __float2bfloat16_rn((0.5f * hi - 0.5f * lowf) * (1.f / 7.5f));
    const float s = __bfloat162float(scale);
    uint32_t codes = 0;
    if (bad != 0.f || isinf(lowf)) {  // bad is 0 or NaN
      low = scale = __ushort_as_bfloat16(0x7fff);
    } else if (s > 0.f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) codes |= uint32_t(code_of(x[j], lowf, s)) << (4 * j);
    }
    uint8_t* sub = at.sub + int64_t(head) * f.block();
    const int row = at.row % kKv4Sub;
    if (is_v) {
      reinterpret_cast<uint32_t*>(sub + f.vc() + row * (f.dv / 2))[f.vword(word)] = codes;
      if (word % 8 == 0) {
        reinterpret_cast<__nv_bfloat16*>(sub + f.vs())[row * f.gv() + group] = scale;
        reinterpret_cast<__nv_bfloat16*>(sub + f.vl())[group * kKv4Sub + row] = low;
      }
    } else {
      reinterpret_cast<uint32_t*>(sub + f.kc() + row * (f.dqk / 2))[f.kword(word)] = codes;
      if (word % 8 == 0) {
        __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(sub + f.kp()) + row * 2 * f.gk() + group;
        p[0] = scale;
        p[f.gk()] = low;
      }
      if (word == 0 && c.weights)
        c.weights[(int64_t(at.page) * c.hkv + head) * CP_KV4_PAGE + at.row] =
            w ? __ldg(w + int64_t(head) * src_rows + src) : 0.f;
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4Cache c, const Kv4Format f, const int32_t* cu,
                                                            const int32_t* start, int64_t tokens, E* k, E* v,
                                                            int per_block) {
  const int nk = f.dqk / 8, nv = f.dv / 8, words = c.hkv * (nk + nv);
  const int64_t t0 = int64_t(blockIdx.x) * per_block;
  const int n = int(min(int64_t(per_block), tokens - t0)) * words;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int64_t t = t0 + i / words;
    int r = i % words;
    Place at;
    if (!find_place(c, f, cu, start, t, &at)) continue;
    const bool is_v = r >= c.hkv * nk;
    if (is_v) r -= c.hkv * nk;
    const int per = is_v ? nv : nk, head = r / per, word = r % per, group = word / 8;
    const uint8_t* sub = at.sub + int64_t(head) * f.block();
    const int row = at.row % kKv4Sub;
    uint32_t codes;
    float s, low;
    if (is_v) {
      codes = reinterpret_cast<const uint32_t*>(sub + f.vc() + row * (f.dv / 2))[f.vword(word)];
      s = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(sub + f.vs())[row * f.gv() + group]);
      low = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(sub + f.vl())[group * kKv4Sub + row]);
    } else {
      codes = reinterpret_cast<const uint32_t*>(sub + f.kc() + row * (f.dqk / 2))[f.kword(word)];
      const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(sub + f.kp()) + row * 2 * f.gk() + group;
      s = __bfloat162float(p[0]);
      low = __bfloat162float(p[f.gk()]);
    }
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaf(s, float((codes >> (4 * j)) & 15u), low);
    store8(is_v ? v + (t * c.hkv * nv + r) * 8 : k + (t * c.hkv * nk + r) * 8, x);
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

// One CTA per (sequence, kv head): the slots to keep, in order.  The key of
// the last slot that is kept is found digit by digit (8 bits a pass, counted
// in shared memory); a second walk writes the slots out in order.
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const Kv4Cache c, const int32_t* lengths,
                                                                 int32_t budget, int32_t recent, int32_t* new_lengths,
                                                                 int32_t* kept) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix, s_need;
  __shared__ uint32_t warp_sum[kSelThreads / 32];
  const int b = blockIdx.x / c.hkv, h = blockIdx.x - b * c.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = kv4_length(c, lengths, b);
  const int keep = min(n, budget);
  int32_t* out = kept + (int64_t(b) * c.hkv + h) * budget;
  if (h == 0 && tid == 0) new_lengths[b] = keep;
  for (int i = keep + tid; i < budget; i += kSelThreads) out[i] = -1;
  if (n <= budget) {
    for (int i = tid; i < n; i += kSelThreads) out[i] = i;
    return;
  }
  const int m = n - recent;        // slots ranked by weight
  int need = budget - recent;      // of which this many stay (need < m)
  auto key_at = [&](int j) -> uint32_t {
    const int page = kv4_page(c, b, j / CP_KV4_PAGE);
    return page < 0 ? 0u : rank_key(__ldg(c.weights + (int64_t(page) * c.hkv + h) * CP_KV4_PAGE + j % CP_KV4_PAGE));
  };
  uint32_t prefix = 0;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int j = tid; j < m; j += kSelThreads) {
        const uint32_t key = key_at(j);
        if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t left = uint32_t(need);
        int d = 255;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        s_prefix = prefix | (uint32_t(d) << shift);
        s_need = left;
      }
      __syncthreads();
      prefix = s_prefix;
      need = int(s_need);
      __syncthreads();
    }
  }
  // slots above the key stay, and the first `need` of those that equal it
  int written = 0, equal = 0;
  const bool none = budget == recent;
  for (int j0 = 0; j0 < n; j0 += kSelThreads) {
    const int j = j0 + tid;
    uint32_t key = 0;
    const bool ranked = j < m;
    if (ranked && !none) key = key_at(j);
    const bool above = j < n && (!ranked || (!none && key > prefix)), same = ranked && !none && key == prefix;
    const uint32_t ma = __ballot_sync(0xffffffffu, above), ms = __ballot_sync(0xffffffffu, same);
    if (lane == 0) warp_sum[warp] = uint32_t(__popc(ma)) | (uint32_t(__popc(ms)) << 16);
    __syncthreads();
    int ba = 0, bs = 0, ta = 0, ts = 0;
    for (int i = 0; i < kSelThreads / 32; ++i) {
      const int a = int(warp_sum[i] & 0xffffu), s = int(warp_sum[i] >> 16);
      if (i < warp) ba += a, bs += s;
      ta += a;
      ts += s;
    }
    const uint32_t below = (1u << lane) - 1u;
    const int a_before = ba + __popc(ma & below), s_before = equal + bs + __popc(ms & below);
    if (above || (same && s_before < need)) {
      const int at = written + a_before + max(0, min(s_before, need) - min(equal, need));
      out[at] = j;
    }
    written += ta + max(0, min(equal + ts, need) - min(equal, need));
    equal += ts;
    __syncthreads();
  }
}

// A warp per sub-block of 32 kept slots: codes, parameters and weights move as they are.
__global__ void __launch_bounds__(kThreads) kv4_move_kernel(const Kv4Cache c, const Kv4Cache to, const Kv4Format f,
                                                            int32_t budget, const int32_t* new_lengths,
                                                            const int32_t* kept) {
  const int lane = threadIdx.x & 31;
  const int subs = (budget + kKv4Sub - 1) / kKv4Sub;
  const int64_t unit = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit >= int64_t(subs) * c.num_seqs * c.hkv) return;
  const int64_t bh = unit / subs;
  const int u = int(unit - bh * subs), b = int(bh / c.hkv), h = int(bh - int64_t(b) * c.hkv);
  const int n = __ldg(new_lengths + b), first = u * kKv4Sub;
  if (first >= n) return;
  const int dst_page = kv4_page(to, b, first / CP_KV4_PAGE);
  if (dst_page < 0) return;
  const int64_t dst_block = int64_t(dst_page) * c.hkv + h;
  uint8_t* dst = to.pages + dst_block * f.block() + (first % CP_KV4_PAGE) / kKv4Sub * f.sub();
  // where this lane's slot comes from: sub-block (or null) and row
  const uint8_t* src = nullptr;
  int row = 0;
  if (first + lane < n) {
    const int j = __ldg(kept + bh * budget + first + lane);
    const int page = kv4_page(c, b, j / CP_KV4_PAGE);
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
    for (int i = lane; i < kKv4Sub * per; i += 32) {  // kKv4Sub * per is a multiple of 32: the warp stays whole
      const int t = i / per, e = i - t * per;
      int r;
      const uint8_t* s = from(t, &r);
      if (s) reinterpret_cast<T*>(dst + off)[i] = __ldg(reinterpret_cast<const T*>(s + off) + r * per + e);
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

// Tokens a CTA of append or read takes: about one word a thread, whole tokens.
static int tokens_per_block(const Kv4Cache& c, int dqk, int dv) {
  const int words = c.hkv * (dqk + dv) / 8;
  return words >= kThreads ? 1 : kThreads / words;
}

cudaError_t launch_kv4_append(const Kv4Cache& c, int dqk, int dv, int dtype, const void* k, const void* v,
                              const float* w, int64_t src_rows, const int32_t* rows, const int32_t* cu,
                              const int32_t* start, int64_t tokens, cudaStream_t st) {
  const int per = tokens_per_block(c, dqk, dv);
  const unsigned grid = unsigned((tokens + per - 1) / per);
  if (dtype == CP_DT_BF16)
    kv4_append_kernel<<<grid, kThreads, 0, st>>>(c, Kv4Format(dqk, dv), static_cast<const __nv_bfloat16*>(k),
                                                 static_cast<const __nv_bfloat16*>(v), w, src_rows, rows, cu, start,
                                                 tokens, per);
  else
    kv4_append_kernel<<<grid, kThreads, 0, st>>>(c, Kv4Format(dqk, dv), static_cast<const float*>(k),
                                                 static_cast<const float*>(v), w, src_rows, rows, cu, start, tokens,
                                                 per);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Cache& c, int dqk, int dv, int dtype, const int32_t* cu, const int32_t* start,
                            int64_t tokens, void* k, void* v, cudaStream_t st) {
  const int per = tokens_per_block(c, dqk, dv);
  const unsigned grid = unsigned((tokens + per - 1) / per);
  if (dtype == CP_DT_BF16)
    kv4_read_kernel<<<grid, kThreads, 0, st>>>(c, Kv4Format(dqk, dv), cu, start, tokens,
                                               static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), per);
  else
    kv4_read_kernel<<<grid, kThreads, 0, st>>>(c, Kv4Format(dqk, dv), cu, start, tokens, static_cast<float*>(k),
                                               static_cast<float*>(v), per);
  return cudaGetLastError();
}

cudaError_t launch_kv4_evict(const Kv4Cache& c, int dqk, int dv, const int32_t* lengths, int32_t budget,
                             int32_t recent, const Kv4Cache& to, int32_t* new_lengths, int32_t* kept,
                             cudaStream_t st) {
  kv4_select_kernel<<<unsigned(c.num_seqs) * unsigned(c.hkv), kSelThreads, 0, st>>>(c, lengths, budget, recent,
                                                                                    new_lengths, kept);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t units = int64_t((budget + kKv4Sub - 1) / kKv4Sub) * c.num_seqs * c.hkv;
  const int64_t grid = (units + kThreads / 32 - 1) / (kThreads / 32);
  kv4_move_kernel<<<unsigned(grid), kThreads, 0, st>>>(c, to, Kv4Format(dqk, dv), budget, new_lengths, kept);
  return cudaGetLastError();
}

}  // namespace cpattn
