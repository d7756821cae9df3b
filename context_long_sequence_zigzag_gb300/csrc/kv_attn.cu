// kv_attn.cu — attention of the newest tokens over the paged cache in the
// model's own type: a CTA a query row, a warp a slot at a time, on CUDA cores.
#include <cmath>

#include "kv.cuh"

namespace cpattn {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename E>
__global__ void __launch_bounds__(32 * kWarps) kv_attn_kernel(const KvAttnArgs a, const int dqk, const int dv) {
  __shared__ float om[kWarps][128], ml[kWarps][2];
  const int row = blockIdx.x, hq = a.c.hq, h = row % hq, t = row / hq % a.n_q, b = row / (hq * a.n_q);
  const int kvh = a.c.inter ? h % a.c.hkv : h / (hq / a.c.hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = kv_length(__ldg(a.lengths + b), int64_t(a.c.max_pages) << a.c.page_shift, a.c.err) - (a.n_q - 1 - t);
  const E* q = static_cast<const E*>(a.q) + int64_t(row) * dqk;
  float qr[6], o[4] = {}, m = -INFINITY, l = 0.f;
  for (int i = 0; i < 6; ++i) qr[i] = 32 * i < dqk ? to_f(q[32 * i + lane]) * a.c.scale : 0.f;
  int seen = 0;
  for (int j = warp; j < n; j += kWarps) {
    const int32_t pg = kv_page(__ldg(a.c.table + int64_t(b) * a.c.max_pages + (j >> a.c.page_shift)), a.c.num_pages, a.c.err);
    if (pg < 0) continue;
    seen = 1;
    const int64_t r = ((int64_t(pg) * a.c.hkv + kvh) << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
    float s = 0.f;
    for (int i = 0; i < 6; ++i)
      if (32 * i < dqk) s = fmaf(qr[i], to_f(static_cast<const E*>(a.c.k)[r * dqk + 32 * i + lane]), s);
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.f : top, f = expf(m - ref), p = expf(s - ref);
    m = top;
    l = l * f + p;
    for (int i = 0; i < 4; ++i)
      if (32 * i < dv) o[i] = fmaf(p, to_f(static_cast<const E*>(a.c.v)[r * dv + 32 * i + lane]), o[i] * f);
  }
  seen = __syncthreads_or(seen);
  for (int i = 0; i < 4; ++i) om[warp][32 * i + lane] = o[i];
  if (lane == 0) ml[warp][0] = m, ml[warp][1] = l;
  __syncthreads();
  float top = -INFINITY, sum = 0.f, out = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][0]);
  const float ref = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kWarps; ++w) {
    const float f = expf(ml[w][0] - ref);
    sum += f * ml[w][1];
    if (threadIdx.x < dv) out += f * om[w][threadIdx.x];
  }
  if (threadIdx.x < dv) {
    const float x = seen ? out / sum : 0.f;
    const int64_t at = int64_t(row) * dv + threadIdx.x;
    if (a.o_f32) static_cast<float*>(a.o)[at] = x;
    else static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(x);
  }
  if (threadIdx.x == 0) a.lse[int64_t(h) * a.c.num_seqs * a.n_q + b * a.n_q + t] = ref + logf(sum);
}

}  // namespace

size_t kv_attn_workspace(const cp_kv_t*, int32_t) { return 256; }

cudaError_t launch_kv_attn(const KvAttnArgs& a, int dqk, int dv, int dtype, cudaStream_t st) {
  const unsigned rows = unsigned(a.c.num_seqs) * a.n_q * a.c.hq;
  if (dtype == CP_DT_BF16) kv_attn_kernel<__nv_bfloat16><<<rows, 32 * kWarps, 0, st>>>(a, dqk, dv);
  else kv_attn_kernel<float><<<rows, 32 * kWarps, 0, st>>>(a, dqk, dv);
  return cudaGetLastError();
}

}  // namespace cpattn
