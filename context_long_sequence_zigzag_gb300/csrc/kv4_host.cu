// kv4_host.cu — entry points of the 4-bit key/value cache: checks of the
// descriptor and the arguments, then the launches.  Lengths, offsets and
// tables stay on the device (the kernels check what they index), so every
// call can be captured into a graph and replayed with new ones.
#include <cmath>

#include <nvtx3/nvToolsExt.h>

#include "kv4.cuh"

namespace cpattn {
namespace {

struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

cp_status_t check_dims(int32_t d_qk, int32_t d_v) {
  if (d_qk < 1 || d_v < 1) return CP_ERR_INVALID_ARG;
  if ((d_qk != 64 && d_qk != 128 && d_qk != 192) || (d_v != 64 && d_v != 128)) return CP_ERR_UNSUPPORTED;
  return CP_OK;
}

cp_status_t check_cache(const cp_kv4_t* c) {
  if (c == nullptr) return CP_ERR_INVALID_ARG;
  if (c->num_seqs < 0 || c->hq < 1 || c->hkv < 1 || c->hq % c->hkv != 0) return CP_ERR_INVALID_ARG;
  if (c->gqa != CP_GQA_BLOCKED && c->gqa != CP_GQA_INTERLEAVED) return CP_ERR_INVALID_ARG;
  if (c->dtype != CP_DT_F32 && c->dtype != CP_DT_BF16) return CP_ERR_INVALID_ARG;
  if (!(c->scale > 0.f) || !std::isfinite(c->scale)) return CP_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->max_pages < 0) return CP_ERR_INVALID_ARG;
  const cp_status_t st = check_dims(c->d_qk, c->d_v);
  if (st != CP_OK) return st;
  // slots, units of work and rows of a call stay below 2^31
  if (c->num_seqs > CP_KV4_MAX_SEQS || c->hq > 1024 || c->max_pages > (1 << 24)) return CP_ERR_UNSUPPORTED;
  if (int64_t(c->num_seqs) * c->hkv * c->max_pages > (int64_t(1) << 29)) return CP_ERR_UNSUPPORTED;
  if (!aligned(c->pages, 16) || !aligned(c->page_table, 4)) {
    // an empty cache needs neither
    if (c->num_seqs > 0 && c->max_pages > 0) return CP_ERR_INVALID_ARG;
  }
  if (c->weights != nullptr && !aligned(c->weights, 16)) return CP_ERR_INVALID_ARG;
  return CP_OK;
}

Kv4Cache device_cache(const cp_kv4_t* c) {
  Kv4Cache d{};
  d.pages = static_cast<uint8_t*>(c->pages);
  d.weights = c->weights;
  d.table = c->page_table;
  d.num_seqs = c->num_seqs;
  d.hq = c->hq;
  d.hkv = c->hkv;
  d.num_pages = c->num_pages;
  d.max_pages = c->max_pages;
  d.inter = c->gqa == CP_GQA_INTERLEAVED;
  d.scale = c->scale;
  d.err = device_error_word();
  return d;
}

cp_status_t check_queries(const cp_kv4_t* c, int32_t n_q) {
  if (n_q < 1) return CP_ERR_INVALID_ARG;
  if (n_q > CP_KV4_MAX_QUERIES) return CP_ERR_UNSUPPORTED;
  if (kv4_attn_units(c, n_q) > INT32_MAX) return CP_ERR_UNSUPPORTED;
  return CP_OK;
}

cp_status_t done(cudaError_t e) { return e == cudaSuccess ? CP_OK : CP_ERR_CUDA; }

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" {

cp_status_t cp_kv4_block_bytes(int32_t d_qk, int32_t d_v, size_t* bytes) {
  if (bytes == nullptr) return CP_ERR_INVALID_ARG;
  const cp_status_t st = check_dims(d_qk, d_v);
  if (st == CP_OK) *bytes = size_t(Kv4Format(d_qk, d_v).block());
  return st;
}

cp_status_t cp_kv4_validate(const cp_kv4_t* c) { return check_cache(c); }

cp_status_t cp_kv4_workspace_size(const cp_kv4_t* c, int32_t n_q, int32_t accumulate, size_t* bytes) {
  if (bytes == nullptr || (accumulate != 0 && accumulate != 1)) return CP_ERR_INVALID_ARG;
  cp_status_t st = check_cache(c);
  if (st == CP_OK) st = check_queries(c, n_q);
  if (st == CP_OK) *bytes = kv4_attn_workspace(c, n_q, accumulate);
  return st;
}

cp_status_t cp_kv4_append(const cp_kv4_t* c, const void* k, const void* v, const float* w, int64_t src_rows,
                          const int32_t* rows, const int32_t* cu, const int32_t* start, int64_t tokens,
                          cp_stream_t stream) {
  CallRange range_("cp_kv4_append");
  const cp_status_t st = check_cache(c);
  if (st != CP_OK) return st;
  if (tokens < 0 || tokens > INT32_MAX || src_rows < 0 || src_rows > INT32_MAX) return CP_ERR_INVALID_ARG;
  if (rows == nullptr && src_rows < tokens) return CP_ERR_INVALID_ARG;
  if (tokens == 0 || c->num_seqs == 0) return CP_OK;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu, 4) || !aligned(start, 4)) return CP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(w) & 3) || (reinterpret_cast<uintptr_t>(rows) & 3)) return CP_ERR_INVALID_ARG;
  return done(launch_kv4_append(device_cache(c), c->d_qk, c->d_v, c->dtype, k, v, w, src_rows, rows, cu, start, tokens,
                                reinterpret_cast<cudaStream_t>(stream)));
}

cp_status_t cp_kv4_read(const cp_kv4_t* c, const int32_t* cu, const int32_t* start, int64_t tokens, void* k, void* v,
                        cp_stream_t stream) {
  CallRange range_("cp_kv4_read");
  const cp_status_t st = check_cache(c);
  if (st != CP_OK) return st;
  if (tokens < 0 || tokens > INT32_MAX) return CP_ERR_INVALID_ARG;
  if (tokens == 0 || c->num_seqs == 0) return CP_OK;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu, 4) || !aligned(start, 4)) return CP_ERR_INVALID_ARG;
  return done(launch_kv4_read(device_cache(c), c->d_qk, c->d_v, c->dtype, cu, start, tokens, k, v,
                              reinterpret_cast<cudaStream_t>(stream)));
}

cp_status_t cp_kv4_attn(const cp_kv4_t* c, int32_t n_q, const void* q, const int32_t* lengths, void* o, int32_t o_f32,
                        float* lse, int32_t accumulate, void* ws, size_t ws_bytes, cp_stream_t stream) {
  CallRange range_("cp_kv4_attn");
  cp_status_t st = check_cache(c);
  if (st == CP_OK) st = check_queries(c, n_q);
  if (st != CP_OK) return st;
  if ((accumulate != 0 && accumulate != 1) || (o_f32 != 0 && o_f32 != 1)) return CP_ERR_INVALID_ARG;
  if (accumulate && c->weights == nullptr) return CP_ERR_INVALID_ARG;
  if (c->num_seqs == 0) return CP_OK;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(lengths, 4)) return CP_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || ws_bytes < kv4_attn_workspace(c, n_q, accumulate)) return CP_ERR_WORKSPACE;
  Kv4AttnArgs a{};
  a.c = device_cache(c);
  a.n_q = n_q;
  a.q = q;
  a.lengths = lengths;
  a.o = o;
  a.o_f32 = o_f32 || c->dtype == CP_DT_F32;
  a.lse = lse;
  a.accumulate = accumulate;
  a.ws = static_cast<char*>(ws);
  return done(launch_kv4_attn(a, c->d_qk, c->d_v, c->dtype, reinterpret_cast<cudaStream_t>(stream)));
}

cp_status_t cp_kv4_evict(const cp_kv4_t* c, const int32_t* lengths, int32_t budget, int32_t recent, const cp_kv4_t* to,
                         int32_t* new_lengths, int32_t* kept, cp_stream_t stream) {
  CallRange range_("cp_kv4_evict");
  cp_status_t st = check_cache(c);
  if (st == CP_OK) st = check_cache(to);
  if (st != CP_OK) return st;
  if (to->num_seqs != c->num_seqs || to->hkv != c->hkv || to->d_qk != c->d_qk || to->d_v != c->d_v)
    return CP_ERR_INVALID_ARG;
  if (budget < 1 || recent < 0 || recent > budget || int64_t(budget) > int64_t(to->max_pages) * CP_KV4_PAGE)
    return CP_ERR_INVALID_ARG;
  if (c->num_seqs == 0) return CP_OK;
  if (c->weights == nullptr || to->weights == nullptr) return CP_ERR_INVALID_ARG;
  if (!aligned(lengths, 4) || !aligned(new_lengths, 4) || !aligned(kept, 4)) return CP_ERR_INVALID_ARG;
  // every CTA reads the lengths, one writes the new ones
  if (lengths < new_lengths + c->num_seqs && new_lengths < lengths + c->num_seqs) return CP_ERR_INVALID_ARG;
  if (c->page_table == to->page_table && c->pages == to->pages) return CP_ERR_INVALID_ARG;  // reads what it writes
  return done(launch_kv4_evict(device_cache(c), c->d_qk, c->d_v, lengths, budget, recent, device_cache(to),
                               new_lengths, kept, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
