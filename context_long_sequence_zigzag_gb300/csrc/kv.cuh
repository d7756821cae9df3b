// kv.cuh — the key/value cache in the model's own type, rotary positions and
// the pages that sequences share: kernel arguments and launchers
// (include/cp_attn.h describes the layouts and the calls).
#pragma once

#include <cuda_bf16.h>

#include "internal.h"

namespace cpattn {

// Sites of the device error word (0x300 | site), those of the 4-bit cache among them.
enum : int32_t { kKvPage = 1, kKvLength = 2, kKvSlot = 3, kKvRow = 4, kKvNoPage = 5, kKvAxis = 6 };

__device__ __forceinline__ void kv_error(int32_t* err, int32_t site) {
  if (err) atomicCAS(err, 0, 0x300 | site);
}

// What the kernels need of a cp_kv_t.
struct KvCache {
  void* k;
  void* v;
  const int32_t* table;
  int32_t num_seqs, hq, hkv, num_pages, max_pages;
  int32_t page_shift;  // log2 of the page size
  int32_t inter;       // interleaved GQA
  float scale;
  int32_t* err;
};

// A length that the table can hold (else recorded and clamped).
__device__ __forceinline__ int32_t kv_length(int32_t n, int64_t most, int32_t* err) {
  if (n >= 0 && n <= most) return n;
  kv_error(err, kKvLength);
  return n < 0 ? 0 : int32_t(most);
}

// Page of a table, or -1 (recorded) where it names none of the pool's.
__device__ __forceinline__ int32_t kv_page(int32_t p, int32_t num_pages, int32_t* err) {
  if (p >= 0 && p < num_pages) return p;
  kv_error(err, kKvPage);
  return -1;
}

// What the kernels need of a cp_rope_t.
struct Rope {
  const uint64_t* turns;
  const int32_t* axis;
  int32_t first, pairs, axes, adjacent;
  float factor;
};

struct RopeArgs {
  Rope r;
  const int32_t* positions;
  int32_t pos_stride;
  int64_t tokens;
  int32_t d, inverse;
  int32_t heads[2];  // of q and k
  const void* in[2];
  void* out[2];
  int32_t* err;
};

struct KvAppendArgs {
  KvCache c;
  Rope r;  // pairs = 0: none
  int32_t d_qk, d_v;
  const void* k;
  const void* v;
  int64_t src_rows, tokens;
  const int32_t* rows;
  const int32_t* cu;
  const int32_t* start;
  const int32_t* positions;
  int32_t pos_stride;
};

struct KvAttnArgs {
  KvCache c;
  int32_t n_q;
  const void* q;
  const int32_t* lengths;
  void* o;
  int32_t o_f32;
  float* lse;
  char* ws;
};

int sm_count();  // of the current device
cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_kv_append(const KvAppendArgs& a, int dtype, cudaStream_t st);
size_t kv_attn_workspace(const cp_kv_t* c, int32_t n_q);
// units of work of the longest sequences that the table can hold
int64_t kv_attn_units(const cp_kv_t* c, int32_t n_q);
cudaError_t launch_kv_attn(const KvAttnArgs& a, int dqk, int dv, int dtype, cudaStream_t st);

// ---- pages ----
struct PageBuffers {
  int32_t n;
  int32_t num_pages[2];  // of the pool read and the pool written
  char* from[CP_PAGES_MAX_BUFFERS];
  char* to[CP_PAGES_MAX_BUFFERS];
  int64_t bytes[CP_PAGES_MAX_BUFFERS];
};

// A batch's table, as the page calls take it.
struct PageTable {
  int32_t num_seqs, max_pages;
  const int32_t* table;
  const int32_t* lengths;
};

size_t pages_workspace(int32_t num_pages, int32_t num_seqs);
cudaError_t launch_pages_reserve(int32_t num_pages, int32_t page_size, int32_t* refs, PageTable t, int32_t* table,
                                 const int32_t* extra, int32_t* counts, int32_t* err, cudaStream_t st);
cudaError_t launch_pages_fork(const PageBuffers& b, int32_t page_size, int32_t* refs, PageTable t, int32_t new_seqs,
                              int32_t new_max_pages, const int32_t* parents, int32_t* new_table, int32_t* new_lengths,
                              int32_t* counts, char* ws, int32_t* err, cudaStream_t st);
cudaError_t launch_pages_compact(const PageBuffers& b, int32_t page_size, int32_t* refs, PageTable t,
                                 int32_t* new_table, int32_t* moved, int32_t* counts, char* ws, int32_t* err,
                                 cudaStream_t st);
cudaError_t launch_pages_copy(const PageBuffers& b, int32_t n, const int32_t* src, const int32_t* dst, int32_t* err,
                              cudaStream_t st);

}  // namespace cpattn
