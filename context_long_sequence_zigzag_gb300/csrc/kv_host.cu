// kv_host.cu — entry points of rotary positions, the key/value cache in the
// model's own type and the pages that sequences share: checks of descriptors
// and arguments, then the launches.  Positions, lengths and tables stay on the
// device (the kernels check what they index), so every call can be captured
// into a graph and replayed with new ones.
#include <cmath>

#include <nvtx3/nvToolsExt.h>

#include "kv.cuh"

namespace cpattn {
namespace {

struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Bytes [a, a + n) and [b, b + m) have some in common.
bool overlap(const void* a, int64_t n, const void* b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return n > 0 && m > 0 && x < y + uintptr_t(m) && y < x + uintptr_t(n);
}

cp_status_t done(cudaError_t e) { return e == cudaSuccess ? CP_OK : CP_ERR_CUDA; }

// A rope that turns channels of heads of d.
cp_status_t check_rope(const cp_rope_t* r, int32_t d, int32_t pos_stride, bool positions) {
  if (r == nullptr) return CP_ERR_INVALID_ARG;
  if (r->dims < 2 || r->dims % 2 || r->first < 0 || r->axes < 1) return CP_ERR_INVALID_ARG;
  if (r->dims > CP_ROPE_MAX_DIMS || r->axes > CP_ROPE_MAX_AXES) return CP_ERR_UNSUPPORTED;
  if (r->first > d || r->dims > d - r->first) return CP_ERR_INVALID_ARG;
  if (r->pairing != CP_ROPE_HALVES && r->pairing != CP_ROPE_ADJACENT) return CP_ERR_INVALID_ARG;
  if (!std::isfinite(r->factor)) return CP_ERR_INVALID_ARG;
  if (positions && pos_stride < r->axes) return CP_ERR_INVALID_ARG;
  if (!aligned(r->turns, 8) || (reinterpret_cast<uintptr_t>(r->axis) & 3)) return CP_ERR_INVALID_ARG;
  return CP_OK;
}
Rope device_rope(const cp_rope_t* r) {
  return {r->turns, r->axis, r->first, r->dims / 2, r->axes, r->pairing == CP_ROPE_ADJACENT, r->factor};
}

int page_shift(int32_t n) {
  for (int s = 4; s <= 7; ++s)
    if (n == 1 << s) return s;
  return -1;
}

cp_status_t check_cache(const cp_kv_t* c) {
  if (c == nullptr) return CP_ERR_INVALID_ARG;
  if (c->num_seqs < 0 || c->hq < 1 || c->hkv < 1 || c->hq % c->hkv != 0) return CP_ERR_INVALID_ARG;
  if (c->gqa != CP_GQA_BLOCKED && c->gqa != CP_GQA_INTERLEAVED) return CP_ERR_INVALID_ARG;
  if (c->dtype != CP_DT_F32 && c->dtype != CP_DT_BF16) return CP_ERR_INVALID_ARG;
  if (!(c->scale > 0.f) || !std::isfinite(c->scale)) return CP_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->max_pages < 0 || c->page_size < 1 || c->d_qk < 1 || c->d_v < 1) return CP_ERR_INVALID_ARG;
  if ((c->d_qk != 64 && c->d_qk != 128 && c->d_qk != 192) || (c->d_v != 64 && c->d_v != 128)) return CP_ERR_UNSUPPORTED;
  if (page_shift(c->page_size) < 0) return CP_ERR_UNSUPPORTED;
  // slots and rows of a call, and rows of the pool (TMA coordinates), stay below 2^31, the scale times log2(e) in range
  if (c->scale > 1e38f) return CP_ERR_UNSUPPORTED;
  if (c->num_seqs > CP_KV4_MAX_SEQS || c->hq > 1024) return CP_ERR_UNSUPPORTED;
  if (int64_t(c->max_pages) * c->page_size > (1 << 30)) return CP_ERR_UNSUPPORTED;
  if (int64_t(c->num_pages) * c->hkv * c->page_size > INT32_MAX) return CP_ERR_UNSUPPORTED;
  if (c->num_seqs > 0 && c->max_pages > 0) {  // (an empty cache needs none of them)
    if (!aligned(c->page_table, 4)) return CP_ERR_INVALID_ARG;
    if (c->num_pages > 0 && (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16))) return CP_ERR_INVALID_ARG;
  }
  return CP_OK;
}

KvCache device_cache(const cp_kv_t* c) {
  KvCache d{};
  d.k = c->k_pages;
  d.v = c->v_pages;
  d.table = c->page_table;
  d.num_seqs = c->num_seqs;
  d.hq = c->hq;
  d.hkv = c->hkv;
  d.num_pages = c->num_pages;
  d.max_pages = c->max_pages;
  d.page_shift = page_shift(c->page_size);
  d.inter = c->gqa == CP_GQA_INTERLEAVED;
  d.scale = c->scale;
  d.err = device_error_word();
  return d;
}

cp_status_t check_queries(const cp_kv_t* c, int32_t n_q) {
  if (n_q < 1) return CP_ERR_INVALID_ARG;
  return n_q > CP_KV4_MAX_QUERIES || kv_attn_units(c, n_q) > INT32_MAX ? CP_ERR_UNSUPPORTED : CP_OK;
}

cp_status_t check_pool(const cp_pages_t* p) {
  if (p == nullptr) return CP_ERR_INVALID_ARG;
  if (p->num_pages < 0 || p->page_size < 1 || p->num_buffers < 0) return CP_ERR_INVALID_ARG;
  if (p->num_pages > 1 << 24 || p->num_buffers > CP_PAGES_MAX_BUFFERS) return CP_ERR_UNSUPPORTED;
  if (p->num_pages > 0 && !aligned(p->refs, 4)) return CP_ERR_INVALID_ARG;
  if (p->num_buffers > 0 && (p->base == nullptr || p->bytes == nullptr)) return CP_ERR_INVALID_ARG;
  for (int i = 0; i < p->num_buffers; ++i) {
    if (p->bytes[i] < 16 || p->bytes[i] % 16) return CP_ERR_INVALID_ARG;
    if (p->bytes[i] > int64_t(1) << 34) return CP_ERR_UNSUPPORTED;
    if (p->num_pages > 0 && !aligned(p->base[i], 16)) return CP_ERR_INVALID_ARG;
  }
  return CP_OK;
}

cp_status_t check_table(const cp_pages_t* p, int32_t num_seqs, int32_t max_pages) {
  if (num_seqs < 0 || max_pages < 0) return CP_ERR_INVALID_ARG;
  if (num_seqs > CP_KV4_MAX_SEQS) return CP_ERR_UNSUPPORTED;
  return int64_t(max_pages) * p->page_size > INT32_MAX ? CP_ERR_UNSUPPORTED : CP_OK;
}

PageBuffers device_buffers(const cp_pages_t* from, const cp_pages_t* to) {
  PageBuffers b{};
  b.n = from->num_buffers;
  b.num_pages[0] = from->num_pages;
  b.num_pages[1] = to->num_pages;
  for (int i = 0; i < b.n; ++i) {
    b.from[i] = static_cast<char*>(from->base[i]);
    b.to[i] = static_cast<char*>(to->base[i]);
    b.bytes[i] = from->bytes[i];
  }
  return b;
}

// 1 / (2 pi) in 192 bits behind the point: pi = 3.243F6A88 85A308D3 13198A2E 03707344 A4093822 299F31D0 ... in hex.
constexpr uint64_t kInvTwoPi[3] = {0x28BE60DB9391054Aull, 0x7F09D5F47D4D3770ull, 0x36D8A5664F10E410ull};

// x / (2 pi) modulo 1 in units of 2^-64, rounded down (0 <= x < 2^32).
uint64_t turns_of(double x) {
  int e;
  const double f = std::frexp(x, &e);  // x = f 2^e, 1/2 <= f < 1
  const uint64_t m = uint64_t(std::ldexp(f, 53));
  e -= 53;  // x = m 2^e
  // m / (2 pi), 64 bits before and 192 behind the point
  uint64_t w[4] = {};  // w[0]: the integer part
  unsigned __int128 carry = 0;
  for (int i = 2; i >= 0; --i) {
    carry += static_cast<unsigned __int128>(m) * kInvTwoPi[i];
    w[i + 1] = uint64_t(carry);
    carry >>= 64;
  }
  w[0] = uint64_t(carry);
  // the 64 bits that 2^e moves right behind the point: bits -e - 63 .. -e - 0 relative to it
  const int at = 64 + e;  // first wanted bit, counted from the top of w[0]
  uint64_t r = 0;
  for (int i = 0; i < 64; ++i) {
    const int bit = at + i;
    if (bit < 0 || bit >= 256) continue;
    r |= (w[bit / 64] >> (63 - bit % 64) & 1) << (63 - i);
  }
  return r;
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" {

cp_status_t cp_rope_turns(const double* inv_freq, int32_t pairs, uint64_t* turns) {
  if (pairs < 0 || (pairs > 0 && (inv_freq == nullptr || turns == nullptr))) return CP_ERR_INVALID_ARG;
  for (int i = 0; i < pairs; ++i)
    if (!(std::fabs(inv_freq[i]) < 4294967296.0)) return CP_ERR_INVALID_ARG;
  for (int i = 0; i < pairs; ++i) {
    const uint64_t t = inv_freq[i] == 0.0 ? 0 : turns_of(std::fabs(inv_freq[i]));
    turns[i] = inv_freq[i] < 0.0 ? 0 - t : t;
  }
  return CP_OK;
}

cp_status_t cp_rope(const cp_rope_t* rope, int64_t tokens, const int32_t* positions, int32_t pos_stride, int32_t d,
                    int32_t dtype, int32_t hq, const void* q, void* q_out, int32_t hkv, const void* k, void* k_out,
                    int32_t inverse, cp_stream_t stream) {
  CallRange range_("cp_rope");
  if (tokens < 0 || tokens > INT32_MAX || d < 1 || hq < 0 || hkv < 0) return CP_ERR_INVALID_ARG;
  if (dtype != CP_DT_F32 && dtype != CP_DT_BF16) return CP_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return CP_ERR_INVALID_ARG;
  const int64_t elt = dtype == CP_DT_BF16 ? 2 : 4;
  if (d * elt % 16) return CP_ERR_INVALID_ARG;
  if (d > 1024 || hq > 1024 || hkv > 1024) return CP_ERR_UNSUPPORTED;
  const cp_status_t st = check_rope(rope, d, pos_stride, true);
  if (st != CP_OK) return st;
  if (tokens == 0 || hq + hkv == 0) return CP_OK;
  if (!aligned(positions, 4)) return CP_ERR_INVALID_ARG;
  RopeArgs a{};
  a.r = device_rope(rope);
  a.positions = positions;
  a.pos_stride = pos_stride;
  a.tokens = tokens;
  a.d = d;
  a.inverse = inverse;
  a.heads[0] = hq, a.heads[1] = hkv;
  a.in[0] = q, a.in[1] = k;
  a.out[0] = q_out, a.out[1] = k_out;
  a.err = device_error_word();
  int64_t bytes[2];
  for (int i = 0; i < 2; ++i) {
    bytes[i] = tokens * a.heads[i] * d * elt;
    if (a.heads[i] && (!aligned(a.in[i], 16) || !aligned(a.out[i], 16))) return CP_ERR_INVALID_ARG;
  }
  // an output is its input, or apart from everything
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (!(i == j && a.out[i] == a.in[i]) && overlap(a.out[i], bytes[i], a.in[j], bytes[j])) return CP_ERR_INVALID_ARG;
  if (overlap(a.out[0], bytes[0], a.out[1], bytes[1])) return CP_ERR_INVALID_ARG;
  return done(launch_rope(a, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

cp_status_t cp_kv_validate(const cp_kv_t* c) { return check_cache(c); }

cp_status_t cp_kv_workspace_size(const cp_kv_t* c, int32_t n_q, size_t* bytes) {
  if (bytes == nullptr) return CP_ERR_INVALID_ARG;
  cp_status_t st = check_cache(c);
  if (st == CP_OK) st = check_queries(c, n_q);
  if (st == CP_OK) *bytes = kv_attn_workspace(c, n_q);
  return st;
}

cp_status_t cp_kv_append(const cp_kv_t* c, const void* k, const void* v, int64_t src_rows, const int32_t* rows,
                         const int32_t* cu, const int32_t* start, int64_t tokens, const cp_rope_t* rope,
                         const int32_t* positions, int32_t pos_stride, cp_stream_t stream) {
  CallRange range_("cp_kv_append");
  cp_status_t st = check_cache(c);
  if (st == CP_OK && rope != nullptr) st = check_rope(rope, c->d_qk, pos_stride, positions != nullptr);
  if (st != CP_OK) return st;
  if (tokens < 0 || tokens > INT32_MAX || src_rows < 0 || src_rows > INT32_MAX) return CP_ERR_INVALID_ARG;
  if (rows == nullptr && src_rows < tokens) return CP_ERR_INVALID_ARG;
  if (tokens == 0 || c->num_seqs == 0) return CP_OK;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu, 4) || !aligned(start, 4)) return CP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(rows) & 3) || (reinterpret_cast<uintptr_t>(positions) & 3)) return CP_ERR_INVALID_ARG;
  KvAppendArgs a{};
  a.c = device_cache(c);
  if (rope != nullptr) a.r = device_rope(rope);
  a.d_qk = c->d_qk, a.d_v = c->d_v;
  a.k = k, a.v = v;
  a.src_rows = src_rows, a.tokens = tokens;
  a.rows = rows;
  a.cu = cu;
  a.start = start;
  a.positions = positions;
  a.pos_stride = pos_stride;
  return done(launch_kv_append(a, c->dtype, reinterpret_cast<cudaStream_t>(stream)));
}

cp_status_t cp_kv_attn(const cp_kv_t* c, int32_t n_q, const void* q, const int32_t* lengths, void* o, int32_t o_f32,
                       float* lse, void* ws, size_t ws_bytes, cp_stream_t stream) {
  CallRange range_("cp_kv_attn");
  cp_status_t st = check_cache(c);
  if (st == CP_OK) st = check_queries(c, n_q);
  if (st != CP_OK) return st;
  if (o_f32 != 0 && o_f32 != 1) return CP_ERR_INVALID_ARG;
  if (c->num_seqs == 0) return CP_OK;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(lengths, 4)) return CP_ERR_INVALID_ARG;
  const size_t need = kv_attn_workspace(c, n_q);
  if (need > 0 && (!aligned(ws, 256) || ws_bytes < need)) return CP_ERR_WORKSPACE;
  KvAttnArgs a{};
  a.c = device_cache(c);
  a.n_q = n_q;
  a.q = q;
  a.lengths = lengths;
  a.o = o;
  a.o_f32 = o_f32 || c->dtype == CP_DT_F32;
  a.lse = lse;
  a.ws = static_cast<char*>(ws);
  return done(launch_kv_attn(a, c->d_qk, c->d_v, c->dtype, reinterpret_cast<cudaStream_t>(stream)));
}

cp_status_t cp_pages_validate(const cp_pages_t* p) { return check_pool(p); }

cp_status_t cp_pages_workspace_size(const cp_pages_t* p, int32_t num_seqs, size_t* bytes) {
  if (bytes == nullptr) return CP_ERR_INVALID_ARG;
  cp_status_t st = check_pool(p);
  if (st == CP_OK) st = check_table(p, num_seqs, 0);
  if (st == CP_OK) *bytes = pages_workspace(p->num_pages, num_seqs);
  return st;
}

cp_status_t cp_pages_reserve(const cp_pages_t* p, int32_t num_seqs, int32_t max_pages, int32_t* table,
                             const int32_t* lengths, const int32_t* extra, int32_t* counts, cp_stream_t stream) {
  CallRange range_("cp_pages_reserve");
  cp_status_t st = check_pool(p);
  if (st == CP_OK) st = check_table(p, num_seqs, max_pages);
  if (st != CP_OK) return st;
  // pages that come and go are summed over the batch in 32 bits, and counted on by the cluster's threads
  if (int64_t(num_seqs) * max_pages > 1 << 30) return CP_ERR_UNSUPPORTED;
  if (!aligned(counts, 4)) return CP_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!aligned(lengths, 4) || !aligned(extra, 4))) return CP_ERR_INVALID_ARG;
  if (num_seqs > 0 && max_pages > 0 && !aligned(table, 4)) return CP_ERR_INVALID_ARG;
  return done(launch_pages_reserve(p->num_pages, p->page_size, p->refs, {num_seqs, max_pages, table, lengths}, table,
                                   extra, counts, device_error_word(), reinterpret_cast<cudaStream_t>(stream)));
}

cp_status_t cp_pages_fork(const cp_pages_t* p, int32_t num_seqs, int32_t max_pages, const int32_t* table,
                          const int32_t* lengths, int32_t new_seqs, int32_t new_max_pages, const int32_t* parents,
                          int32_t* new_table, int32_t* new_lengths, int32_t* counts, void* ws, size_t ws_bytes,
                          cp_stream_t stream) {
  CallRange range_("cp_pages_fork");
  cp_status_t st = check_pool(p);
  if (st == CP_OK) st = check_table(p, num_seqs, max_pages);
  if (st == CP_OK) st = check_table(p, new_seqs, new_max_pages);
  if (st != CP_OK) return st;
  if (!aligned(counts, 4)) return CP_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!aligned(lengths, 4) || (max_pages > 0 && !aligned(table, 4)))) return CP_ERR_INVALID_ARG;
  if (new_seqs > 0 && (!aligned(parents, 4) || !aligned(new_lengths, 4))) return CP_ERR_INVALID_ARG;
  if (new_seqs > 0 && new_max_pages > 0 && !aligned(new_table, 4)) return CP_ERR_INVALID_ARG;
  const int64_t rows = int64_t(num_seqs) * 4, new_rows = int64_t(new_seqs) * 4;
  const int64_t old_bytes = rows * max_pages, new_bytes = new_rows * new_max_pages;
  if (overlap(table, old_bytes, new_table, new_bytes) || overlap(lengths, rows, new_lengths, new_rows) ||
      overlap(parents, new_rows, new_lengths, new_rows))
    return CP_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || ws_bytes < pages_workspace(p->num_pages, num_seqs > new_seqs ? num_seqs : new_seqs))
    return CP_ERR_WORKSPACE;
  return done(launch_pages_fork(device_buffers(p, p), p->page_size, p->refs, {num_seqs, max_pages, table, lengths},
                                new_seqs, new_max_pages, parents, new_table, new_lengths, counts,
                                static_cast<char*>(ws), device_error_word(), reinterpret_cast<cudaStream_t>(stream)));
}

cp_status_t cp_pages_compact(const cp_pages_t* p, int32_t num_seqs, int32_t max_pages, const int32_t* table,
                             const int32_t* lengths, int32_t* new_table, int32_t* moved, int32_t* counts, void* ws,
                             size_t ws_bytes, cp_stream_t stream) {
  CallRange range_("cp_pages_compact");
  cp_status_t st = check_pool(p);
  if (st == CP_OK) st = check_table(p, num_seqs, max_pages);
  if (st != CP_OK) return st;
  if (!aligned(counts, 4) || (p->num_pages > 0 && !aligned(moved, 4))) return CP_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!aligned(lengths, 4) || (max_pages > 0 && (!aligned(table, 4) || !aligned(new_table, 4)))))
    return CP_ERR_INVALID_ARG;
  const int64_t bytes = int64_t(num_seqs) * 4 * max_pages;
  if (table != new_table && overlap(table, bytes, new_table, bytes)) return CP_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || ws_bytes < pages_workspace(p->num_pages, num_seqs)) return CP_ERR_WORKSPACE;
  return done(launch_pages_compact(device_buffers(p, p), p->page_size, p->refs, {num_seqs, max_pages, table, lengths},
                                   new_table, moved, counts, static_cast<char*>(ws), device_error_word(),
                                   reinterpret_cast<cudaStream_t>(stream)));
}

cp_status_t cp_pages_copy(const cp_pages_t* p, const cp_pages_t* to, int32_t n, const int32_t* src, const int32_t* dst,
                          cp_stream_t stream) {
  CallRange range_("cp_pages_copy");
  cp_status_t st = check_pool(p);
  if (st == CP_OK) st = check_pool(to);
  if (st != CP_OK) return st;
  if (n < 0 || p->num_buffers != to->num_buffers) return CP_ERR_INVALID_ARG;
  for (int i = 0; i < p->num_buffers; ++i)
    if (p->bytes[i] != to->bytes[i]) return CP_ERR_INVALID_ARG;
  if (n == 0 || p->num_buffers == 0) return CP_OK;
  if (!aligned(src, 4) || !aligned(dst, 4)) return CP_ERR_INVALID_ARG;
  return done(launch_pages_copy(device_buffers(p, to), n, src, dst, device_error_word(),
                                reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
