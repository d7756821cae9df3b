// kv4.cuh — the 4-bit key/value cache: page format, kernel arguments and
// launchers (include/cp_attn.h describes the format and the calls).
#pragma once

#include <cuda_bf16.h>

#include "internal.h"

namespace cpattn {

constexpr int kKv4Sub = 32;    // tokens of a sub-block, the unit of work
constexpr int kKv4Group = 64;  // channels that share a scale and a low

// Byte offsets inside a sub-block of 32 tokens.
struct Kv4Format {
  int dqk, dv;
  __host__ __device__ constexpr Kv4Format(int dqk_, int dv_) : dqk(dqk_), dv(dv_) {}
  __host__ __device__ constexpr int gk() const { return dqk / kKv4Group; }
  __host__ __device__ constexpr int gv() const { return dv / kKv4Group; }
  __host__ __device__ constexpr int kc() const { return 0; }
  __host__ __device__ constexpr int vc() const { return kc() + kKv4Sub * dqk / 2; }
  __host__ __device__ constexpr int kp() const { return vc() + kKv4Sub * dv / 2; }
  __host__ __device__ constexpr int vs() const { return kp() + kKv4Sub * gk() * 4; }
  __host__ __device__ constexpr int vl() const { return vs() + kKv4Sub * gv() * 2; }
  __host__ __device__ constexpr int sub() const { return vl() + kKv4Sub * gv() * 2; }
  __host__ __device__ constexpr int block() const { return 2 * sub(); }
  // word position of channels 8w .. 8w + 7 in a row
  __host__ __device__ constexpr int kword(int w) const { return (w % 4) * (dqk / 32) + w / 4; }
  __host__ __device__ constexpr int vword(int w) const { return (w % 8) * (dv / 64) + w / 8; }
};

// What the kernels need of a cp_kv4_t.
struct Kv4Cache {
  uint8_t* pages;
  float* weights;
  const int32_t* table;
  int32_t num_seqs, hq, hkv, num_pages, max_pages;
  int32_t inter;  // interleaved GQA
  float scale;
  int32_t* err;
};

// Sites of the device error word (0x300 | site).
enum : int32_t { kKv4Page = 1, kKv4Length = 2, kKv4Slot = 3, kKv4Row = 4 };

__device__ __forceinline__ void kv4_error(const Kv4Cache& c, int32_t site) {
  if (c.err) atomicCAS(c.err, 0, 0x300 | site);
}

// Page of a sequence's slot, or -1 (recorded) where the table names none of the pool's.
__device__ __forceinline__ int32_t kv4_page(const Kv4Cache& c, int b, int32_t page_of_seq) {
  const int32_t p = __ldg(c.table + int64_t(b) * c.max_pages + page_of_seq);
  if (p >= 0 && p < c.num_pages) return p;
  kv4_error(c, kKv4Page);
  return -1;
}

// A length that the table can hold (else recorded and clamped).
__device__ __forceinline__ int32_t kv4_length(const Kv4Cache& c, const int32_t* lengths, int b) {
  const int32_t n = __ldg(lengths + b), most = c.max_pages * CP_KV4_PAGE;
  if (n >= 0 && n <= most) return n;
  kv4_error(c, kKv4Length);
  return n < 0 ? 0 : most;
}

// Sequence b with cu[b] <= t < cu[b + 1], or -1 past the last.
__device__ __forceinline__ int kv4_seq_of(const int32_t* cu, int n, int64_t t) {
  if (n == 0 || t >= __ldg(cu + n)) return -1;
  int lo = 0, hi = n - 1;  // the last b with cu[b] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct Kv4AttnArgs {
  Kv4Cache c;
  int32_t n_q, rows;     // queries a sequence; rows of a kv head: G * n_q
  int32_t row_tiles;     // passes over the cache for those rows
  const void* q;
  const int32_t* lengths;
  void* o;
  int32_t o_f32;
  float* lse;
  int32_t accumulate;
  char* ws;
};

cudaError_t launch_kv4_append(const Kv4Cache& c, int dqk, int dv, int dtype, const void* k, const void* v,
                              const float* w, int64_t src_rows, const int32_t* rows, const int32_t* cu,
                              const int32_t* start, int64_t tokens, cudaStream_t st);
cudaError_t launch_kv4_read(const Kv4Cache& c, int dqk, int dv, int dtype, const int32_t* cu, const int32_t* start,
                            int64_t tokens, void* k, void* v, cudaStream_t st);
cudaError_t launch_kv4_evict(const Kv4Cache& c, int dqk, int dv, const int32_t* lengths, int32_t budget,
                             int32_t recent, const Kv4Cache& to, int32_t* new_lengths, int32_t* kept,
                             cudaStream_t st);
int kv4_sm_count();  // of the current device
size_t kv4_attn_workspace(const cp_kv4_t* c, int32_t n_q, int32_t accumulate);
// units of work of the longest sequences that the table can hold
int64_t kv4_attn_units(const cp_kv4_t* c, int32_t n_q);
// fills in rows and row_tiles
cudaError_t launch_kv4_attn(Kv4AttnArgs a, int dqk, int dv, int dtype, cudaStream_t st);

}  // namespace cpattn
