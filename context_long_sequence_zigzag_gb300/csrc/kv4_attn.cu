// kv4_attn.cu — attention of single tokens (or a few) over the 4-bit cache.
//
// Row (b, t, h) sees slots j < lengths[b] - (n_q - 1 - t):
//   S_j = scale q.K_j,  lse = log sum_j exp(S_j),  o = sum_j exp(S_j - lse) V_j.
// One CTA per row; its warps take the slots in turn, each with a running
// maximum and sum, and are joined at the end.
#include "kv4.cuh"
#include "sm103_ptx.cuh"

namespace cpattn {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ldf(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename E>
__global__ void __launch_bounds__(kWarps * 32) kv4_attn_kernel(const Kv4AttnArgs a, const Kv4Format f) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][128];
  const Kv4Cache& c = a.c;
  const int G = c.hq / c.hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;  // (b, t, h)
  const int h = int(row % c.hq);
  const int64_t bt = row / c.hq;
  const int t = int(bt % a.n_q), b = int(bt / a.n_q);
  const int kvh = c.inter ? h % c.hkv : h / G;
  const int n = kv4_length(c, a.lengths, b) - (a.n_q - 1 - t);
  const E* q = static_cast<const E*>(a.q) + row * f.dqk;
  // lane: channels 8w .. 8w + 7 of word w = lane, lane < d / 8
  float qv[8] = {}, o[8] = {};
  if (lane < f.dqk / 8)
    for (int i = 0; i < 8; ++i) qv[i] = ldf(q + 8 * lane + i);
  auto block_of = [&](int j, int* r) -> const uint8_t* {
    const int page = kv4_page(c, b, j / CP_KV4_PAGE);
    *r = j % kKv4Sub;
    return page < 0 ? nullptr
                    : c.pages + (int64_t(page) * c.hkv + kvh) * f.block() + (j % CP_KV4_PAGE) / kKv4Sub * f.sub();
  };
  auto score = [&](const uint8_t* sub, int r) {
    float x = 0.f;
    if (lane < f.dqk / 8) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(sub + f.kc() + r * (f.dqk / 2))[f.kword(lane)];
      const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(sub + f.kp()) + r * 2 * f.gk() + lane / 8;
      const float s = __bfloat162float(p[0]), lo = __bfloat162float(p[f.gk()]);
      for (int i = 0; i < 8; ++i) x += fmaf(s, float((w >> (4 * i)) & 15u), lo) * qv[i];
    }
    return warp_sum(x) * c.scale;
  };
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < n; j += kWarps) {
    int r;
    const uint8_t* sub = block_of(j, &r);
    if (!sub) continue;
    const float x = score(sub, r);
    const float top = fmaxf(m, x);
    const float keep = m == -INFINITY ? 0.f : expf(m - top), p = x == -INFINITY ? 0.f : expf(x - top);
    m = top;
    l = l * keep + p;
    if (lane < f.dv / 8) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(sub + f.vc() + r * (f.dv / 2))[f.vword(lane)];
      const float s = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(sub + f.vs())[r * f.gv() + lane / 8]);
      const float lo = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(sub + f.vl())[lane / 8 * kKv4Sub + r]);
      for (int i = 0; i < 8; ++i) o[i] = o[i] * keep + p * fmaf(s, float((w >> (4 * i)) & 15u), lo);
    }
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  if (lane < f.dv / 8)
    for (int i = 0; i < 8; ++i) s_o[warp][8 * lane + i] = o[i];
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  for (int w = 0; w < kWarps; ++w) total += s_m[w] == -INFINITY ? 0.f : s_l[w] * expf(s_m[w] - top);
  const float lse = top == -INFINITY ? -INFINITY : top + logf(total);
  if (threadIdx.x == 0) a.lse[int64_t(h) * c.num_seqs * a.n_q + bt] = lse;
  for (int e = threadIdx.x; e < f.dv; e += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += s_m[w] == -INFINITY ? 0.f : s_o[w][e] * expf(s_m[w] - top);
    x = top == -INFINITY ? 0.f : x / total;
    if (a.o_f32) static_cast<float*>(a.o)[row * f.dv + e] = x;
    else static_cast<__nv_bfloat16*>(a.o)[row * f.dv + e] = __float2bfloat16_rn(x);
  }
}

// Every visible slot's probabilities, summed over its head's rows in one
// order and added once.  A warp per slot.
template <typename E>
__global__ void __launch_bounds__(kWarps * 32) kv4_weights_kernel(const Kv4AttnArgs a, const Kv4Format f) {
  const Kv4Cache& c = a.c;
  const int G = c.hq / c.hkv, lane = threadIdx.x & 31;
  const int b = blockIdx.x / c.hkv, kvh = blockIdx.x - b * c.hkv;
  const int n = kv4_length(c, a.lengths, b);
  for (int j = blockIdx.y * kWarps + (threadIdx.x >> 5); j < n; j += gridDim.y * kWarps) {
    const int page = kv4_page(c, b, j / CP_KV4_PAGE);
    if (page < 0) continue;
    const int64_t block = int64_t(page) * c.hkv + kvh;
    const uint8_t* sub = c.pages + block * f.block() + (j % CP_KV4_PAGE) / kKv4Sub * f.sub();
    const int r = j % kKv4Sub;
    float kv[8] = {};
    if (lane < f.dqk / 8) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(sub + f.kc() + r * (f.dqk / 2))[f.kword(lane)];
      const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(sub + f.kp()) + r * 2 * f.gk() + lane / 8;
      const float s = __bfloat162float(p[0]), lo = __bfloat162float(p[f.gk()]);
      for (int i = 0; i < 8; ++i) kv[i] = fmaf(s, float((w >> (4 * i)) & 15u), lo);
    }
    float sum = 0.f;
    for (int t = 0; t < a.n_q; ++t) {
      if (j >= n - (a.n_q - 1 - t)) continue;
      for (int g = 0; g < G; ++g) {
        const int h = c.inter ? g * c.hkv + kvh : kvh * G + g;
        const int64_t bt = int64_t(b) * a.n_q + t;
        float x = 0.f;
        if (lane < f.dqk / 8)
          for (int i = 0; i < 8; ++i) x += kv[i] * ldf(static_cast<const E*>(a.q) + (bt * c.hq + h) * f.dqk + 8 * lane + i);
        sum += expf(warp_sum(x) * c.scale - a.lse[int64_t(h) * c.num_seqs * a.n_q + bt]);
      }
    }
    if (lane == 0) atomicAdd(c.weights + block * CP_KV4_PAGE + j % CP_KV4_PAGE, sum);
  }
}

template <typename E>
cudaError_t launch(const Kv4AttnArgs& a, Kv4Format f, cudaStream_t st) {
  kv4_attn_kernel<E><<<unsigned(a.c.num_seqs) * unsigned(a.n_q) * unsigned(a.c.hq), kWarps * 32, 0, st>>>(a, f);
  if (a.accumulate)
    kv4_weights_kernel<E><<<dim3(unsigned(a.c.num_seqs) * unsigned(a.c.hkv), 64), kWarps * 32, 0, st>>>(a, f);
  return cudaGetLastError();
}

}  // namespace

size_t kv4_attn_workspace(const cp_kv4_t*, int32_t, int32_t) { return 256; }

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, int dqk, int dv, int dtype, cudaStream_t st) {
  return dtype == CP_DT_BF16 ? launch<__nv_bfloat16>(a, Kv4Format(dqk, dv), st) : launch<float>(a, Kv4Format(dqk, dv), st);
}

}  // namespace cpattn
