// kv_attn.cu — attention of the newest tokens over the paged cache in the
// model's own type: o = sum_j p_j v_j, p = softmax(scale q.k), one pass over
// the cache with the running maximum and sum of the softmax.
//
// What bounds it: the cache's bytes, read once (d_qk + d_v elements a slot and
// head, for 2 (d_qk + d_v) G n_q FLOPs).  With the 1 to 16 rows that share a
// head in decoding a tcgen05 tile (64 or 128 rows) would be mostly empty and its
// accumulator a detour through TMEM; warp-level MMAs of 16 rows keep up with the
// copies, with up to 32 rows (8 x 8K, 32/8 heads: 47 to 54 us).  64 rows, which
// they bound (64 us), would fill such a tile; there is no such variant.
//
// Work.  A run is one sequence's slots for one kv head and up to 16, 32 or 64
// of its rows (query heads of the group times new tokens); its tiles are TT
// slots.  All runs' tiles laid end to end (a run's start counts as one more)
// are cut evenly over the CTAs, on the device, from the lengths: a long
// sequence keeps every SM busy, and a captured graph replays with new lengths.
// A cut run's parts go to the workspace and a second kernel joins them, whose
// launch overlaps the first.  Few short sequences take a cluster a run instead.
//
// A CTA: a producer warp looks the pages up and brings tiles of K and V in by
// TMA, 128-byte swizzled panels through a ring of stages; queries come two
// runs ahead.  Four compute warps share every tile: MT of them side by side in
// rows, the others along the slots, each with its own maximum, sum and O, which
// meet once a run, in shared memory.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "kv.cuh"
#include "sm103_ptx.cuh"

namespace cpattn {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_tiled();

namespace {

constexpr int kWarps = 4;  // that compute; the first of four more produces (registers move by four warps)
constexpr int kThreads = 32 * 2 * kWarps;
// Registers a thread: two CTAs an SM start with 128; the producers hand theirs to the computing warps.
constexpr int kLaunchRegs = 128, kComputeRegs = 200, kProducerRegs = 56;
static_assert(kComputeRegs + kProducerRegs == 2 * kLaunchRegs, "what one half takes the other gives");
constexpr int kMostStages = 6;
// Sequences whose lengths the producer warp adds up alone, a lane each, without the other warps' barrier: the first copy
// leaves 0.6 us earlier (1 x 16K 19.0 us, by all warps 19.6).
constexpr int kFewSeqs = 32;
// A cluster of up to eight CTAs a run, in the place of even shares and a second kernel, where the table holds no more
// tokens than this and the clusters fit the GPU at once.  32/8 heads, one sequence of 512 tokens: 8.1 us on the device
// (even shares: 9.4); 8 of 4K: 26.3 us (28.9); 8 ragged ones up to 4K: 20.4 us (21.4) or, of other lengths, 16.0 (12.7);
// one of 4K: 12.5 us (10.7), but 15 us of a host that calls again and again (20), which decides here; one of 8K: 18.4 us
// (13.0).  So a replayed graph pays 2 to 3 us for it near the bound; a table of more columns takes even shares.  Clusters
// of sixteen start 1 us later.  Where they do not fit (fp32, 32 rows of 32/8 heads of 192: one CTA an SM), 5 of 512
// tokens: 36.8 us (23.7), 5 of 4K: 150 us (83).
constexpr int64_t kClusterTokens = 4096;
constexpr float kLog2e = 1.4426950408889634f;
// log2 units: a row's reference maximum follows a new one past this (p stays below 2^8 relative to it, so that most
// tiles leave O as it is)
constexpr float kRescale = 8.f;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
enum : int { kSiteQFull = 0x60, kSiteQEmpty, kSiteKFull, kSiteKEmpty, kSiteVFull, kSiteVEmpty, kSiteJoin, kSiteDrain };

template <typename E_, int DQK_, int DV_, int MT_>
struct Cfg {
  using E = E_;
  static constexpr bool F32 = sizeof(E) == 4;
  static constexpr int DQK = DQK_, DV = DV_, MT = MT_;
  static constexpr int NS = kWarps / MT;       // warps along a tile's slots
  static constexpr int TT_SHIFT = F32 ? 5 : 6, TT = 1 << TT_SHIFT;  // slots of a tile
  static constexpr int TS = TT / NS;           // of a warp
  static constexpr int ROWS = 16 * MT;
  // BF16: the product with V takes the probabilities as two terms of BF16, off by 2^-15 of them instead of 2^-8 (8 x 8K,
  // O in fp32 off by 4.6e-6 of its norm instead of 1.4e-3).  With up to 32 rows the MMAs that this adds lie behind the
  // copies (46.8 -> 47.1 us, 32 rows 52.8 -> 53.7; 1 x 4K 11.7 -> 12.4, 1000 x 100 57 -> 60); 64 rows are bound by MMAs and
  // take one term (63.5 us, with two 85.7).
  static constexpr bool REST = !F32 && MT <= 2;
  static constexpr int KP = DQK * sizeof(E) / 128, VP = DV * sizeof(E) / 128;  // panels of 128 bytes
  static constexpr uint32_t KBYTES = KP * TT * 128, VBYTES = VP * TT * 128;
  static constexpr uint32_t QPITCH = DQK * sizeof(E) + 16;  // (rows of a fragment in different banks)
  static constexpr uint32_t QBYTES = (ROWS * QPITCH + 127) / 128 * 128;
};

struct RunDesc {
  int32_t b, head, row0, len;  // b < 0: no more
  int32_t lo, hi;              // tiles of this part
  int32_t whole, slot;         // whole: no parts to join; otherwise the part's slot
};

struct alignas(16) Tail {  // shared memory behind the stages and queries; the buffer that O is joined in follows
  float m[kWarps][16], l[kWarps][16];
  float2 row[16];  // maximum and sum of a row (one row tile)
  alignas(16) RunDesc run[2];
  int32_t absent[kMostStages];  // pages of a K slot that are outside the pool, a bit each
  int32_t warp_units[2 * kWarps];
  int32_t start_b, start_off, total;
  int abort, drain_abort;
  uint64_t q_full[2], q_empty[2], joined;
  uint64_t k_full[kMostStages], k_empty[kMostStages], v_full[kMostStages], v_empty[kMostStages];
};

// Shared memory of a CTA: two on an SM where two tiles fit then.  What is left holds as many slots of K as of V, or one
// more of K (they come first).
constexpr uint32_t kSmShared = 227 * 1024;
template <typename C>
struct Room {
  static constexpr uint32_t half = (kSmShared - 1024) / 2;  // (1 KiB a CTA is the system's)
  static constexpr uint32_t pair = C::KBYTES + C::VBYTES;
  // queries a run ahead and 8 KiB to join in, or less of both
  static constexpr uint32_t fixed_of(int slots, int floats) {
    return 1024 + (slots + (C::F32 ? 1 : 0)) * C::QBYTES + uint32_t(sizeof(Tail)) + floats * 4;
  }
  static constexpr int q_slots = fixed_of(2, 2048) + 2 * pair <= half ? 2 : 1;
  static constexpr int join_floats = fixed_of(q_slots, 2048) + 2 * pair <= half ? 2048 : 1024;
  static constexpr uint32_t fixed = fixed_of(q_slots, join_floats);
  static constexpr bool two = fixed + 2 * pair <= half;
  static constexpr uint32_t ring = (two ? half : kSmShared) - fixed;
  static constexpr int nv = std::min<uint32_t>(ring / pair, kMostStages);
  static constexpr int nk = nv < kMostStages && nv * pair + C::KBYTES <= ring ? nv + 1 : nv;
  static constexpr uint32_t bytes = fixed + nk * C::KBYTES + nv * C::VBYTES;
  static_assert(nv >= 2, "a ring");
};

struct Params {
  KvAttnArgs a;
  CUtensorMap tk, tv;
  int32_t group, rows, row_tiles;  // G; rows of a kv head; runs they take
  int32_t box_shift;               // log2 of the slots a copy brings: a page's, at most a tile's
  // sequence, head and row tile, number of parts (0: not cut) and first CTA of every run; where there are more runs than
  // CTAs, of the run that is cut behind every CTA
  int4* meta;
  int32_t by_run, join_ctas;
  int32_t cluster;  // 0: shares of all units; otherwise the CTAs of a cluster, which take a run's tiles among them
  float* parts;  // [ctas][2][ROWS][DV + 4]: O, its maximum and sum
};

// units of a sequence's run: its tiles and its start
__device__ __forceinline__ int units_of(int len, int tt) { return (len + tt - 1) / tt + 1; }

// All units cut for n CTAs, none without a unit: each gets `least` of them, the first `more` one more.  (One division of
// 32 bits: the CTA's first copy waits for it.)
struct Share {
  int n, least, more;
  __device__ Share(int total, int ctas) : n(min(ctas, total)), least(n ? total / n : 0), more(total - least * n) {}
  // first unit of a CTA; that of CTA n and those behind it: past the last
  __device__ int first(int cta) const { return cta < n ? least * cta + min(cta, more) : least * n + more; }
  __device__ int cta_of(int unit) const {
    const int x = unit - more * (least + 1);
    return x < 0 ? unit / (least + 1) : more + x / least;
  }
};
__device__ __forceinline__ int warp_sum_up_to(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// x as two terms of 11 bits: the first rounded, of the rest (at most 2^-11 of x) the MMA cuts what is below 2^-10 of
// it.  A NaN stays in the second term whatever becomes of it in the first.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return reinterpret_cast<const uint32_t&>(p);
}

// Two numbers >= 0 as two terms of BF16 each: cut off, and the rest with 2^-20 of the number, so that neither term of a
// number above 0 is 0 (whose product with an infinity would be NaN).
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& high, uint32_t& rest) {
  high = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  rest = pack_bf16(fmaf(a, 1.f + 0x1p-20f, -__uint_as_float(high << 16)),
                   fmaf(b, 1.f + 0x1p-20f, -__uint_as_float(high & 0xffff0000u)));
}

// Tiles lie in panels of 128 bytes a slot, 16-byte pieces swizzled: piece c of slot x is piece (c ^ x) % 8 of its row in
// panel c / 8.  row_of: a lane's row and the low bits of its pieces; piece_of: with the other bits, which are constants.
__device__ __forceinline__ uint32_t row_of(int slot, int low) { return (slot << 7) | (((slot ^ low) & 7) << 4); }
template <int TT>
__device__ __forceinline__ uint32_t piece_of(uint32_t row, int c) {
  return (row ^ ((c & 7) << 4)) + (c >> 3) * (TT * 128);
}

// A row's maximum score (before the scale) and sum: what O is multiplied by, and its lse.  A row that saw nothing (or
// scores of -inf alone) has -inf and 0; a NaN stays one.
__device__ __forceinline__ float inverse_of(float2 ml) { return ml.y == 0.f ? 0.f : 1.f / ml.y; }
__device__ __forceinline__ float lse_of(float2 ml, float scale) {
  return ml.y == 0.f ? -INFINITY : fmaf(ml.x == -INFINITY ? 0.f : ml.x, scale, logf(ml.y));
}

// Where the results of row r of a kv head go: row of o, entry of lse.
struct RowOf {
  int64_t o, lse;
  __device__ RowOf(const KvAttnArgs& a, int group, int b, int head, int r) {
    const int t = r / group, g = r - t * group, h = a.c.inter ? head + g * a.c.hkv : head * group + g;
    o = (int64_t(b) * a.n_q + t) * a.c.hq + h;
    lse = int64_t(h) * a.c.num_seqs * a.n_q + int64_t(b) * a.n_q + t;
  }
};
template <int DV>
__device__ __forceinline__ void store_row(const KvAttnArgs& a, int group, int b, int head, int r, int col, float4 v, float2 ml) {
  const RowOf to(a, group, b, head, r);
  const float inv = inverse_of(ml);
  const int64_t at = to.o * DV + col;
  v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
  if (a.o_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.o) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + at) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  if (col == 0) a.lse[to.lse] = lse_of(ml, a.c.scale);
}

// Every thread of a cluster; what was written before is visible behind it.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
  uint32_t x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(addr), "r"(rank));
  return x;
}

template <typename C>
__global__ void __launch_bounds__(kThreads, 2) kv_attn_kernel(const __grid_constant__ Params p) {
  using E = typename C::E;
  constexpr int TT = C::TT, MT = C::MT, NS = C::NS, DV = C::DV;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (ptx::smem_u32(raw) + 1023) & ~1023u;
  constexpr int NK = Room<C>::nk, NV = Room<C>::nv;
  constexpr int QS = Room<C>::q_slots, kJoinFloats = Room<C>::join_floats;
  const uint32_t values = base + NK * C::KBYTES, queries = values + NV * C::VBYTES;
  const uint32_t low_at = queries + QS * C::QBYTES;  // fp32: the second terms of the run's queries
  Tail& sh = *reinterpret_cast<Tail*>(raw + (low_at + (C::F32 ? C::QBYTES : 0) - ptx::smem_u32(raw)));
  float* const join = reinterpret_cast<float*>(&sh + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const KvCache& c = p.a.c;
  if (!p.cluster) ptx::grid_launch_dependents();  // (the second kernel, which waits)
  const int64_t most = int64_t(c.max_pages) << c.page_shift;
  const int runs = c.hkv * p.row_tiles, cta = blockIdx.x, rank = p.cluster ? cta % p.cluster : 0;
  const bool few = c.num_seqs <= kFewSeqs;  // the producer adds their lengths up by itself
  int32_t few_length = 0;
  if (warp == kWarps) {
    if (few && lane < c.num_seqs) few_length = __ldg(p.a.lengths + lane);
    if (lane == 0) {
      ptx::prefetch_tmap(&p.tk);
      ptx::prefetch_tmap(&p.tv);
      for (int i = 0; i < QS; ++i) {
        ptx::mbar_init(ptx::smem_u32(&sh.q_full[i]), 1);
        ptx::mbar_init(ptx::smem_u32(&sh.q_empty[i]), kWarps);
      }
      for (int i = 0; i < NK; ++i) {
        ptx::mbar_init(ptx::smem_u32(&sh.k_full[i]), 1);
        ptx::mbar_init(ptx::smem_u32(&sh.k_empty[i]), kWarps);
      }
      for (int i = 0; i < NV; ++i) {
        ptx::mbar_init(ptx::smem_u32(&sh.v_full[i]), 1);
        ptx::mbar_init(ptx::smem_u32(&sh.v_empty[i]), kWarps);
      }
      ptx::mbar_init(ptx::smem_u32(&sh.joined), kWarps);
      ptx::fence_barrier_init();
      sh.abort = sh.drain_abort = 0;
    }
  } else if (warp < kWarps) {
    // rows past the last of a run's stay 0
    const uint32_t from = min(C::ROWS, p.rows) * C::QPITCH;
    for (int slot = 0; slot < QS; ++slot)
      for (uint32_t i = from + tid * 16; i + 16 <= C::ROWS * C::QPITCH; i += 32 * kWarps * 16)
        *reinterpret_cast<uint4*>(raw + (queries + slot * C::QBYTES - ptx::smem_u32(raw)) + i) = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();
  }
  if (!p.cluster && !few) {
    // where this CTA's share begins: a thread adds up some sequences in a row
    const int per = (c.num_seqs + kThreads - 1) / kThreads, b0 = min(tid * per, c.num_seqs), b1 = min(b0 + per, c.num_seqs);
    int units = 0;
    for (int b = b0; b < b1; ++b) units += units_of(kv_length(__ldg(p.a.lengths + b), most, c.err), TT) * runs;
    int before = warp_sum_up_to(units, lane);
    if (lane == 31) sh.warp_units[warp] = before;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < 2 * kWarps; ++w) {
      if (w == warp) before += total;
      total += sh.warp_units[w];
    }
    before -= units;
    const int u0 = Share(total, int(gridDim.x)).first(cta);
    if (tid == 0) sh.total = total;
    if (before <= u0 && u0 < before + units) {
      int off = u0 - before, b = b0;
      for (;; ++b) {
        const int y = units_of(kv_length(__ldg(p.a.lengths + b), most, nullptr), TT) * runs;
        if (off < y) break;
        off -= y;
      }
      sh.start_b = b, sh.start_off = off;
    }
  }
  __syncthreads();
  const ptx::WaitCtx ctx{&sh.abort, c.err, kWaitLimitNs};

  if (warp >= kWarps) {
    // ------------------------------------------------------------ producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp > kWarps) {
      if (p.cluster) cluster_meet(), cluster_meet();
      return;
    }
    int ks = 0, kphase = 0, vs = 0, vphase = 0, keys_sent = 0, tiles_sent = 0, runs_sent = 0;
    int4 cut = make_int4(0, 0, 0, 0);
    bool ok = true;
    // this CTA's units u0 .. u1 - 1; the first is unit `off` of sequence b.  (A cluster's CTA: one unit, its part of run
    // `off` of sequence b.)
    int b = 0, off = 0, u0 = 0, u1 = 1;
    Share share(0, 0);
    if (p.cluster) {
      b = cta / p.cluster / runs, off = cta / p.cluster - b * runs;
    } else {
      if (few) {
        const int units = lane < c.num_seqs ? units_of(kv_length(few_length, most, c.err), TT) * runs : 0;
        const int upto = warp_sum_up_to(units, lane);
        share = Share(__shfl_sync(~0u, upto, 31), int(gridDim.x));
        off = share.first(cta) - (upto - units);
        const unsigned here = __ballot_sync(~0u, off >= 0 && off < units);
        b = here ? __ffs(here) - 1 : 0;
        off = __shfl_sync(~0u, off, b);
      } else {
        share = Share(sh.total, int(gridDim.x));
        b = sh.start_b, off = sh.start_off;
      }
      u0 = share.first(cta), u1 = share.first(cta + 1);
    }
    for (int u = u0; u < u1 && ok;) {
      const int len = kv_length(__ldg(p.a.lengths + b), most, p.cluster && rank == 0 ? c.err : nullptr);
      const int tiles = (len + TT - 1) / TT, per_run = tiles + 1;
      int r = off, lo, hi, take = 1;
      bool first = false, whole = false;
      if (p.cluster) {
        lo = tiles * rank / p.cluster, hi = tiles * (rank + 1) / p.cluster;  // (at most kClusterTokens / 32 tiles)
      } else {
        r = off / per_run;
        const int at = off - r * per_run;
        take = min(per_run - at, u1 - u);
        lo = max(at - 1, 0), hi = at + take - 1;
        first = lo == 0, whole = first && hi == tiles;
      }
      if (p.cluster || hi > lo || tiles == 0) {
        const int head = p.row_tiles == 1 ? r : r / p.row_tiles;
        const int row0 = (r - head * p.row_tiles) * C::ROWS, rows = min(C::ROWS, p.rows - row0);
        const int slot = runs_sent % QS;
        if (runs_sent >= QS) ok = ptx::mbar_wait(ptx::smem_u32(&sh.q_empty[slot]), (runs_sent / QS - 1) & 1, kSiteQEmpty, ctx);
        if (!__all_sync(~0u, ok)) { ok = false; break; }
        const uint32_t bar = ptx::smem_u32(&sh.q_full[slot]);
        if (lane == 0) {
          sh.run[slot] = RunDesc{b, head, row0, len, lo, hi, whole, cta * 2 + (first ? 1 : 0)};
          ptx::mbar_arrive_expect_tx(bar, hi > lo ? rows * C::DQK * sizeof(E) : 0);
        }
        __syncwarp();
        if (hi > lo) {
          // pages of the part, 32 at a time, a lane each
          const int32_t* table = c.table + int64_t(b) * c.max_pages;
          const int pages = (len + (1 << c.page_shift) - 1) >> c.page_shift;
          int window = (lo * TT) >> c.page_shift;
          int32_t held = window + lane < pages ? __ldg(table + window + lane) : -1;
          for (int i = lane; i < rows; i += 32) {
            const int t = p.a.n_q == 1 ? 0 : (row0 + i) / p.group, g = row0 + i - t * p.group;
            const int h = c.inter ? head + g * c.hkv : head * p.group + g;
            ptx::bulk_load(queries + slot * C::QBYTES + i * C::QPITCH,
                           static_cast<const E*>(p.a.q) + ((int64_t(b) * p.a.n_q + t) * c.hq + h) * C::DQK,
                           C::DQK * sizeof(E), bar);
          }
          const int boxes = TT >> p.box_shift;
          for (int tile = lo; tile < hi && ok; ++tile) {
            const int e0 = (tile * TT) >> c.page_shift;
            if (e0 + boxes > window + 32) {
              window = e0;
              held = window + lane < pages ? __ldg(table + window + lane) : -1;
            }
            // a lane a copy: a page's part of the tile and a panel of it
            const int box = lane & (boxes - 1), panel = lane >> (C::TT_SHIFT - p.box_shift);
            const int slot0 = tile * TT + (box << p.box_shift);
            int32_t page = __shfl_sync(~0u, held, ((slot0 >> c.page_shift) - window) & 31);
            const bool mine = slot0 < len;
            if (mine) page = kv_page(page, c.num_pages, c.err);
            const unsigned there = __ballot_sync(~0u, panel == 0 && mine && page >= 0);
            const unsigned gone = __ballot_sync(~0u, panel == 0 && mine && page < 0);
            const int row = ((page * c.hkv + head) << c.page_shift) + (slot0 & ((1 << c.page_shift) - 1));
            if (tiles_sent >= NK) ok = ptx::mbar_wait(ptx::smem_u32(&sh.k_empty[ks]), kphase ^ 1, kSiteKEmpty, ctx);
            if (!__all_sync(~0u, ok)) { ok = false; break; }
            const uint32_t kbar = ptx::smem_u32(&sh.k_full[ks]), vbar = ptx::smem_u32(&sh.v_full[vs]);
            if (lane == 0) {
              sh.absent[ks] = int32_t(gone);
              ptx::mbar_arrive_expect_tx(kbar, __popc(there) * (C::KBYTES / TT << p.box_shift));
            }
            __syncwarp();
            const uint32_t in_tile = panel * (TT * 128) + (box << (7 + p.box_shift));
            if (mine && page >= 0 && panel < C::KP)
              ptx::tma_load_3d(base + ks * C::KBYTES + in_tile, &p.tk, kbar, 0, row, panel);
            ++keys_sent;
            if (tiles_sent >= NV) ok = ptx::mbar_wait(ptx::smem_u32(&sh.v_empty[vs]), vphase ^ 1, kSiteVEmpty, ctx);
            if (!__all_sync(~0u, ok)) { ok = false; break; }
            if (lane == 0) ptx::mbar_arrive_expect_tx(vbar, __popc(there) * (C::VBYTES / TT << p.box_shift));
            __syncwarp();
            if (mine && page >= 0 && panel < C::VP)
              ptx::tma_load_3d(values + vs * C::VBYTES + in_tile, &p.tv, vbar, 0, row, panel);
            ++tiles_sent;
            if (++ks == NK) ks = 0, kphase ^= 1;
            if (++vs == NV) vs = 0, vphase ^= 1;
          }
        }
        if (first) {  // (what the second kernel reads; the copies come first)
          const int parts = whole ? 0 : share.cta_of(u + take - (hi + 1) + tiles) - cta + 1;
          const int4 x = make_int4(b, r, parts, cta);
          if (p.by_run && lane == 0) p.meta[b * runs + r] = x;
          if (parts) cut = x;
        }
        ++runs_sent;
      }
      u += take;
      off += take;
      if (!p.cluster && off == per_run * runs) ++b, off = 0;
    }
    if (lane == 0) {
      if (ok) {
        const int slot = runs_sent % QS;
        if (runs_sent < QS || ptx::mbar_wait(ptx::smem_u32(&sh.q_empty[slot]), (runs_sent / QS - 1) & 1, kSiteQEmpty, ctx)) {
          sh.run[slot].b = -1;
          ptx::mbar_arrive(ptx::smem_u32(&sh.q_full[slot]));
        }
      }
      if (!p.by_run && !p.cluster) p.meta[cta] = cut;
      // no copy is in flight when the CTA's shared memory goes to the next one (computing warps that gave up did not wait)
      const ptx::WaitCtx drain{&sh.drain_abort, c.err, kWaitLimitNs};
      for (int i = max(keys_sent - NK, 0); i < keys_sent; ++i)
        ptx::mbar_wait(ptx::smem_u32(&sh.k_full[i % NK]), i / NK & 1, kSiteDrain, drain);
      for (int i = max(tiles_sent - NV, 0); i < tiles_sent; ++i)
        ptx::mbar_wait(ptx::smem_u32(&sh.v_full[i % NV]), i / NV & 1, kSiteDrain, drain);
      for (int i = max(runs_sent - QS, 0); i < runs_sent; ++i)
        if (!ok) ptx::mbar_wait(ptx::smem_u32(&sh.q_full[i % QS]), i / QS & 1, kSiteDrain, drain);
    }
    __syncwarp();
    if (p.cluster) cluster_meet(), cluster_meet();
    return;
  }

  // -------------------------------------------------------------- compute
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
  const int mt = warp % MT, slice = warp / MT;
  const int first_slot = slice * C::TS;  // of this warp in a tile
  const int r0 = lane >> 2, quad = lane & 3;
  const float cs = c.scale * kLog2e;
  int ks = 0, kphase = 0, vs = 0, vphase = 0, join_phase = 0;
  bool ok = true;
  auto meet = [&] {
    __syncwarp();
    const uint32_t bar = ptx::smem_u32(&sh.joined);
    if (lane == 0) ptx::mbar_arrive(bar);
    ok = __all_sync(~0u, ptx::mbar_wait(bar, join_phase, kSiteJoin, ctx));
    join_phase ^= 1;
  };
  for (int run = 0; ok; ++run) {
    const int qslot = run % QS;
    ok = ptx::mbar_wait(ptx::smem_u32(&sh.q_full[qslot]), run / QS & 1, kSiteQFull, ctx);
    ok = __all_sync(~0u, ok);
    if (!ok) break;
    const RunDesc d = sh.run[qslot];
    if (d.b < 0) break;
    const uint32_t q_lane = (mt * 16 + (lane & 7) + (lane & 8)) * C::QPITCH + (lane >> 4) * 16;
    const uint32_t q_at = queries + qslot * C::QBYTES + q_lane;
    uint32_t qf[C::F32 ? 1 : C::DQK / 16][4];
    if constexpr (C::F32) {
      // both terms once a run: the first in place
      if (d.lo < d.hi) {
        for (int i = slice * 32 + lane; i < 16 * (C::DQK / 4); i += NS * 32) {
          const uint32_t off = (mt * 16 + i / (C::DQK / 4)) * C::QPITCH + i % (C::DQK / 4) * 16;
          uint4* const at = reinterpret_cast<uint4*>(raw + (queries + qslot * C::QBYTES + off - ptx::smem_u32(raw)));
          uint4 x = *at, y;
          split(__uint_as_float(x.x), x.x, y.x);
          split(__uint_as_float(x.y), x.y, y.y);
          split(__uint_as_float(x.z), x.z, y.z);
          split(__uint_as_float(x.w), x.w, y.w);
          *at = x;
          *reinterpret_cast<uint4*>(raw + (low_at + off - ptx::smem_u32(raw))) = y;
        }
        meet();
        if (!ok) break;
      }
    } else {
#pragma unroll
      for (int k = 0; k < C::DQK / 16; ++k) ptx::ldmatrix_x4(qf[k], q_at + k * 32);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.q_empty[qslot]));
    }
    // slots that this lane's two rows see
    int see[2], query[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = d.row0 + mt * 16 + r0 + 8 * i;
      query[i] = row / p.group;
      see[i] = row < p.rows ? d.len - (p.a.n_q - 1 - query[i]) : 0;
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[DV / 8][4];
#pragma unroll
    for (int i = 0; i < DV / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

    for (int tile = d.lo; tile < d.hi; ++tile) {
      const uint32_t kt = base + ks * C::KBYTES, vt = values + vs * C::VBYTES;
      ok = __all_sync(~0u, ptx::mbar_wait(ptx::smem_u32(&sh.k_full[ks]), kphase, kSiteKFull, ctx));
      if (!ok) break;
      const int absent = sh.absent[ks];
      constexpr int NB = C::TS / 8;  // blocks of 8 slots
      float s[NB][4];
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
      if constexpr (C::F32) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const uint32_t keys = kt + row_of(first_slot + 8 * i + (lane & 7), lane >> 3);
          float low[4][4] = {};  // the products with lower terms, in four chains, added in the end
#pragma unroll 4
          for (int k = 0; k < C::DQK / 16; ++k) {  // two steps of 8 channels
            uint32_t kf[4];
            ptx::ldmatrix_x4(kf, piece_of<TT>(keys, 4 * k));
            float high[4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t ah[4], al[4], bh[2], bl[2];
              ptx::ldmatrix_x4(ah, q_at + k * 64 + x * 32);
              ptx::ldmatrix_x4(al, low_at + q_lane + k * 64 + x * 32);
#pragma unroll
              for (int j = 0; j < 2; ++j) split(__uint_as_float(kf[2 * x + j]), bh[j], bl[j]);
              ptx::mma_1688(low[2 * x], ah, bl[0], bl[1]);
              ptx::mma_1688(low[2 * x + 1], al, bh[0], bh[1]);
              if (x == 0) ptx::mma_1688_first(high, ah, bh[0], bh[1]);
              else ptx::mma_1688(high, ah, bh[0], bh[1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] += high[j];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] += (low[0][j] + low[1][j]) + (low[2][j] + low[3][j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NB; i += 2) {
          const uint32_t keys = kt + row_of(first_slot + 8 * i + (lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);
#pragma unroll
          for (int k = 0; k < C::DQK / 16; ++k) {
            uint32_t kf[4];
            ptx::ldmatrix_x4(kf, piece_of<TT>(keys, 2 * k));
            ptx::mma_16816(s[i], qf[k], kf[0], kf[1]);
            ptx::mma_16816(s[i + 1], qf[k], kf[2], kf[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.k_empty[ks]));
      if (++ks == NK) ks = 0, kphase ^= 1;
      // what not every row sees
      const int tile0 = tile * TT + first_slot;
      const bool masked = (tile + 1) * TT > d.len - (p.a.n_q - 1) || absent;
      if (masked) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int x = first_slot + 8 * i + 2 * quad + (j & 1);
            if (tile * TT + x >= see[j >> 1] || (absent >> (x >> p.box_shift) & 1)) s[i][j] = -INFINITY;
          }
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) top[j >> 1] = fmaxf(top[j >> 1], s[i][j]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 1));
        top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 2));
      }
      if (__any_sync(~0u, (top[0] - m[0]) * cs > kRescale || (top[1] - m[1]) * cs > kRescale)) {
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float next = fmaxf(m[x], top[x]);
          f[x] = next == -INFINITY ? 1.f : ptx::ex2((m[x] - next) * cs);
          m[x] = next;
          l[x] *= f[x];
        }
#pragma unroll
        for (int i = 0; i < DV / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][j] *= f[j >> 1];
      }
      const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = ptx::ex2((s[i][j] - ref[j >> 1]) * cs);  // (that of the reference: exactly 1, however large the score)
          l[j >> 1] += s[i][j];
        }

      ok = __all_sync(~0u, ptx::mbar_wait(ptx::smem_u32(&sh.v_full[vs]), vphase, kSiteVFull, ctx));
      if (!ok) break;
      // O += P V.  GUARD: slots from `end` on and absent ones count as 0 whatever they hold.  ONE: rows of one query only.
      auto product = [&](auto guard, auto one, int end, int only) {
        constexpr bool GUARD = decltype(guard)::value, ONE = decltype(one)::value;
        auto seen = [&](int x) { return tile * TT + x < end && !(absent >> (x >> p.box_shift) & 1); };
        auto add = [&](float (&acc)[4], auto&& f) {
          if constexpr (ONE) {
            float t[4] = {acc[0], acc[1], acc[2], acc[3]};
            f(t);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (query[j >> 1] == only) acc[j] = t[j];
          } else {
            f(acc);
          }
        };
        auto prob = [&](float x, int j) { return !ONE || query[j >> 1] == only ? x : 0.f; };
        if constexpr (C::F32) {
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const int x = first_slot + 8 * i + 2 * quad;  // the MMA's k = quad and quad + 4: slots x and x + 1
            uint32_t ah[4], al[4];
            split(prob(s[i][0], 0), ah[0], al[0]);
            split(prob(s[i][2], 2), ah[1], al[1]);
            split(prob(s[i][1], 1), ah[2], al[2]);
            split(prob(s[i][3], 3), ah[3], al[3]);
            const bool in0 = !GUARD || seen(x), in1 = !GUARD || seen(x + 1);
            const uint32_t v0 = vt + row_of(x, r0 >> 2) + (r0 & 3) * 4, v1 = vt + row_of(x + 1, r0 >> 2) + (r0 & 3) * 4;
#pragma unroll
            for (int nb = 0; nb < DV / 8; ++nb) {
              float v[2];
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0]) : "r"(piece_of<TT>(v0, 2 * nb)) : "memory");
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[1]) : "r"(piece_of<TT>(v1, 2 * nb)) : "memory");
              if (!in0) v[0] = 0.f;
              if (!in1) v[1] = 0.f;
              uint32_t bh[2], bl[2];
              split(v[0], bh[0], bl[0]);
              split(v[1], bh[1], bl[1]);
              add(o[nb], [&](float (&acc)[4]) {
                float t[4];
                ptx::mma_1688_first(t, ah, bl[0], bl[1]);
                ptx::mma_1688(t, al, bh[0], bh[1]);
                ptx::mma_1688(t, ah, bh[0], bh[1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] += t[j];
              });
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < NB; i += 2) {
            uint32_t a[4], rest[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int j = 2 * (y & 1);
              const float x0 = prob(s[i + y / 2][j], j), x1 = prob(s[i + y / 2][j + 1], j + 1);
              if constexpr (C::REST) split_bf16(x0, x1, a[y], rest[y]);
              else a[y] = pack_bf16(x0, x1);
            }
            uint32_t mask[2] = {~0u, ~0u};
            if constexpr (GUARD) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int x = first_slot + 8 * (i + y) + 2 * quad;
                mask[y] = (seen(x) ? 0xffffu : 0u) | (seen(x + 1) ? 0xffff0000u : 0u);
              }
            }
            const uint32_t vals = vt + row_of(first_slot + 8 * i + (lane & 7) + (lane & 8), lane >> 4);
#pragma unroll
            for (int nb = 0; nb < DV / 8; nb += 2) {
              uint32_t vf[4];
              ptx::ldmatrix_x4_trans(vf, piece_of<TT>(vals, nb));
              if constexpr (GUARD) vf[0] &= mask[0], vf[1] &= mask[1], vf[2] &= mask[0], vf[3] &= mask[1];
#pragma unroll
              for (int y = 0; y < 2; ++y)
                add(o[nb + y], [&](float (&acc)[4]) {
                  if constexpr (C::REST) ptx::mma_16816(acc, rest, vf[2 * y], vf[2 * y + 1]);
                  ptx::mma_16816(acc, a, vf[2 * y], vf[2 * y + 1]);
                });
            }
          }
        }
      };
      if (!masked) {
        product(std::false_type{}, std::false_type{}, 0, 0);
      } else {
        // 0 times a value that is not finite is not 0: slots that only later queries see are looked at first
        bool bad = false;
        const int from = max(d.len - (p.a.n_q - 1), tile0), to = min(d.len, tile0 + C::TS);
        for (int x = from; x < to; ++x)
          for (int i = lane; i < DV * int(sizeof(E)) / 16; i += 32) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(piece_of<TT>(vt + row_of(x - tile * TT, 0), i))
                         : "memory");
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              bad = bad || (w[j] & 0x7f800000u) == 0x7f800000u;
              if (!C::F32) bad = bad || (w[j] & 0x7f80u) == 0x7f80u;
            }
          }
        if (!__any_sync(~0u, bad)) {
          product(std::true_type{}, std::false_type{}, d.len, 0);
        } else {
          for (int t = 0; t < p.a.n_q; ++t) product(std::true_type{}, std::true_type{}, d.len - (p.a.n_q - 1 - t), t);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.v_empty[vs]));
      if (++vs == NV) vs = 0, vphase ^= 1;
    }
    if (!ok) break;
    if constexpr (C::F32) {
      ptx::fence_proxy_async_smem();  // (written here, and next by a copy)
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.q_empty[qslot]));
    }

    // ---- the warps along the slots meet
    const int rows = min(C::ROWS, p.rows - d.row0);
    // where the parts of a run that is not whole go (a cluster's: where its tiles were)
    float* const parts = p.cluster ? reinterpret_cast<float*>(raw + (base - ptx::smem_u32(raw)))
                                   : p.parts + int64_t(d.slot) * C::ROWS * (DV + 4);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(~0u, l[x], 1);
      l[x] += __shfl_xor_sync(~0u, l[x], 2);
    }
    if (NS > 1 || p.cluster) {  // (and nobody reads tiles any more)
      if (quad == 0) {
#pragma unroll
        for (int x = 0; x < 2; ++x) sh.m[warp][r0 + 8 * x] = m[x], sh.l[warp][r0 + 8 * x] = l[x];
      }
      meet();
      if (!ok) break;
    }
    if constexpr (NS > 1) {
      float f[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float all = m[x], sum = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) all = fmaxf(all, sh.m[i * MT + mt][r0 + 8 * x]);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const float y = sh.l[i * MT + mt][r0 + 8 * x];
          sum += all == -INFINITY ? y : y * ptx::ex2((sh.m[i * MT + mt][r0 + 8 * x] - all) * cs);
        }
        f[x] = all == -INFINITY ? 1.f : ptx::ex2((m[x] - all) * cs);
        m[x] = all, l[x] = sum;
        if (MT == 1 && warp == 0 && quad == 0) sh.row[r0 + 8 * x] = make_float2(all, sum);
      }
#pragma unroll
      for (int i = 0; i < DV / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] *= f[j >> 1];
    }
    if constexpr (MT == 1) {
      // O by columns, as many at a time as there is room for; all threads add
      const int held = rows <= 4 ? 4 : rows <= 8 ? 8 : 16, cols = min(DV, kJoinFloats / kWarps / held);
      for (int c0 = 0; c0 < DV; c0 += cols) {
#pragma unroll
        for (int i = 0; i < DV / 8; ++i)
          if (8 * i >= c0 && 8 * i < c0 + cols) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (r0 + 8 * x < held)
                *reinterpret_cast<float2*>(&join[(warp * held + r0 + 8 * x) * cols + 8 * i - c0 + 2 * quad]) =
                    make_float2(o[i][2 * x], o[i][2 * x + 1]);
          }
        meet();
        if (!ok) break;
        for (int i = tid; i < rows * cols / 4; i += 32 * kWarps) {
          const int row = i / (cols / 4), col = (i - row * (cols / 4)) * 4;
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < NS; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(&join[(k * held + row) * cols + col]);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
          }
          const float2 ml = sh.row[row];
          if (d.whole) {
            store_row<DV>(p.a, p.group, d.b, d.head, d.row0 + row, c0 + col, sum, ml);
          } else {
            float* to = parts + row * (DV + 4);
            *reinterpret_cast<float4*>(to + c0 + col) = sum;
            if (c0 + col == 0) *reinterpret_cast<float2*>(to + DV) = ml;
          }
        }
        meet();
        if (!ok) break;
      }
    } else {
      // many rows: a row's first warp adds what the other one (if there is one) leaves in shared memory, and stores (all
      // threads adding, as above: 64 rows of 8 x 8K 66 us instead of 63, of 4 x 8K and d 192 40 us instead of 34)
      if constexpr (NS == 2) {
        constexpr int cols = kJoinFloats / (MT * 16) < DV ? kJoinFloats / (MT * 16) : DV;
#pragma unroll
        for (int c0 = 0; c0 < DV; c0 += cols) {
#pragma unroll
          for (int i = c0 / 8; i < (c0 + cols) / 8; ++i)
            if (slice == 1) {
#pragma unroll
              for (int x = 0; x < 2; ++x)
                *reinterpret_cast<float2*>(&join[(mt * 16 + r0 + 8 * x) * cols + 8 * i - c0 + 2 * quad]) =
                    make_float2(o[i][2 * x], o[i][2 * x + 1]);
            }
          meet();
          if (slice == 0) {
#pragma unroll
            for (int i = c0 / 8; i < (c0 + cols) / 8; ++i)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float2 v = *reinterpret_cast<const float2*>(&join[(mt * 16 + r0 + 8 * x) * cols + 8 * i - c0 + 2 * quad]);
                o[i][2 * x] += v.x, o[i][2 * x + 1] += v.y;
              }
          }
          meet();
        }
        if (!ok) break;
      }
      if (slice == 0) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = mt * 16 + r0 + 8 * x;
          if (row >= rows) continue;
          const float2 ml = make_float2(m[x], l[x]);
          const RowOf at(p.a, p.group, d.b, d.head, d.row0 + row);
          const float inv = inverse_of(ml);
          float* const part = parts + row * (DV + 4);
#pragma unroll
          for (int i = 0; i < DV / 8; ++i) {
            const int col = 8 * i + 2 * quad;
            const float2 v = make_float2(o[i][2 * x], o[i][2 * x + 1]);
            if (!d.whole) *reinterpret_cast<float2*>(part + col) = v;
            else if (p.a.o_f32)
              *reinterpret_cast<float2*>(static_cast<float*>(p.a.o) + at.o * DV + col) = make_float2(v.x * inv, v.y * inv);
            else
              *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.a.o) + at.o * DV + col) = pack_bf16(v.x * inv, v.y * inv);
          }
          if (quad == 0) {
            if (d.whole) p.a.lse[at.lse] = lse_of(ml, c.scale);
            else *reinterpret_cast<float2*>(part + DV) = ml;
          }
        }
      }
    }
  }
  if (!p.cluster) return;
  // the run's parts, each in its CTA's shared memory: a CTA joins some of the rows' pieces of four channels
  cluster_meet();
  const int run = blockIdx.x / p.cluster, b = run / runs, r = run - b * runs, head = r / p.row_tiles;
  const int row0 = (r - head * p.row_tiles) * C::ROWS, rows = min(C::ROWS, p.rows - row0);
  for (int i = tid * p.cluster + rank; i < rows * (DV / 4) && ok; i += 32 * kWarps * p.cluster) {
    const int row = i / (DV / 4), col = (i - row * (DV / 4)) * 4;
    const uint32_t at = base + row * (DV + 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = -INFINITY, sum = 0.f;
#pragma unroll 4
    for (int k = 0; k < p.cluster; ++k) {
      float2 ml;
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(ml.x), "=f"(ml.y) : "r"(in_cta(at + DV * 4, k)) : "memory");
      top = fmaxf(top, ml.x);
    }
#pragma unroll 4
    for (int k = 0; k < p.cluster; ++k) {
      float2 ml;
      float4 x;
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(ml.x), "=f"(ml.y) : "r"(in_cta(at + DV * 4, k)) : "memory");
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                   : "r"(in_cta(at + col * 4, k))
                   : "memory");
      const float f = top == -INFINITY ? 1.f : ptx::ex2((ml.x - top) * cs);
      sum = fmaf(f, ml.y, sum);
      v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
    }
    store_row<DV>(p.a, p.group, b, head, row0 + row, col, v, make_float2(top, sum));
  }
  cluster_meet();  // (nobody leaves while its part may still be read)
}


// A cut run's parts: one at the end of a CTA's share, the others at the heads of those that follow it.  A CTA joins
// `rows_a_cta` rows of a run, W / rows_a_cta warps a row.
template <typename C, int W>
__global__ void __launch_bounds__(32 * W) kv_join_kernel(const __grid_constant__ Params p, const int rows_a_cta) {
  constexpr int DV = C::DV, V = DV / 32;
  __shared__ float2 ml_of[W];
  __shared__ __align__(16) float acc_of[W][DV];
  ptx::grid_wait_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 cut = __ldcg(p.meta + blockIdx.x);
  // (a CTA that gave up waiting has left no plan)
  const int ctas = p.join_ctas;
  if (cut.z <= 0 || cut.w < 0 || cut.z > ctas - cut.w || cut.x < 0 || cut.x >= p.a.c.num_seqs || cut.y < 0 ||
      cut.y >= p.a.c.hkv * p.row_tiles)
    return;
  const int across = W / rows_a_cta, row = blockIdx.y * rows_a_cta + warp / across;
  const int head = cut.y / p.row_tiles, r = (cut.y - head * p.row_tiles) * C::ROWS + row;
  const bool mine = row < C::ROWS && r < p.rows;
  const float cs = p.a.c.scale * kLog2e;
  float acc[V] = {}, top = -INFINITY, sum = 0.f;
  auto add = [&](float2 ml, const float (&x)[V]) {
    const float next = fmaxf(top, ml.x);
    const float f = next == -INFINITY ? 1.f : ptx::ex2((top - next) * cs), g = next == -INFINITY ? 1.f : ptx::ex2((ml.x - next) * cs);
    top = next;
    sum = fmaf(sum, f, g * ml.y);
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = fmaf(acc[j], f, g * x[j]);
  };
  if (mine) {
    constexpr int U = 4;  // parts in flight
    for (int i0 = warp % across; i0 < cut.z; i0 += U * across) {
      float2 ml[U];
      float x[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * across;
        if (i >= cut.z) continue;
        const float* from = p.parts + (int64_t(i == 0 ? cut.w * 2 + 1 : (cut.w + i) * 2) * C::ROWS + row) * (DV + 4);
        ml[u] = __ldcg(reinterpret_cast<const float2*>(from + DV));
        if constexpr (V == 4) *reinterpret_cast<float4*>(x[u]) = __ldcg(reinterpret_cast<const float4*>(from) + lane);
        else *reinterpret_cast<float2*>(x[u]) = __ldcg(reinterpret_cast<const float2*>(from) + lane);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * across < cut.z) add(ml[u], x[u]);
    }
  }
  if (lane == 0) ml_of[warp] = make_float2(top, sum);
#pragma unroll
  for (int j = 0; j < V; ++j) acc_of[warp][lane * V + j] = acc[j];
  __syncthreads();
  if (!mine || warp % across) return;
  for (int w = 1; w < across; ++w) {
    float x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = acc_of[warp + w][lane * V + j];
    add(ml_of[warp + w], x);
  }
  const KvCache& c = p.a.c;
  const RowOf to(p.a, p.group, cut.x, head, r);
  const float inv = inverse_of(make_float2(top, sum));
  const int64_t at = to.o * DV + lane * V;
#pragma unroll
  for (int j = 0; j < V; j += 2) {
    if (p.a.o_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.a.o) + at + j) = make_float2(acc[j] * inv, acc[j + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.a.o) + at + j) = pack_bf16(acc[j] * inv, acc[j + 1] * inv);
  }
  if (lane == 0) p.a.lse[to.lse] = lse_of(make_float2(top, sum), c.scale);
}

// Panels of 128 bytes of the rows of a pool.
bool make_map(CUtensorMap* map, const void* pages, bool f32, int64_t rows, int d, int box) {
  EncodeTiledFn enc = get_encode_tiled();
  if (enc == nullptr) return false;
  const int elt = f32 ? 4 : 2, wide = 128 / elt;
  const cuuint64_t dim[3] = {cuuint64_t(wide), cuuint64_t(rows), cuuint64_t(d / wide)};
  const cuuint64_t stride[2] = {cuuint64_t(d * elt), 128};
  const cuuint32_t size[3] = {cuuint32_t(wide), cuuint32_t(box), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(pages),
             dim, stride, size, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// f(Cfg) of a call's kernel.
template <typename E, int DQK, int DV, typename F>
auto with_rows(int rows_a_run, F f) {
  if (rows_a_run == 16) return f(Cfg<E, DQK, DV, 1>{});
  if constexpr (sizeof(E) == 2)
    if (rows_a_run == 64) return f(Cfg<E, DQK, DV, 4>{});
  return f(Cfg<E, DQK, DV, 2>{});
}
template <typename E, typename F>
auto with_dims(int dqk, int dv, int rows_a_run, F f) {
  switch (dqk * 1000 + dv) {
    case 64064: return with_rows<E, 64, 64>(rows_a_run, f);
    case 64128: return with_rows<E, 64, 128>(rows_a_run, f);
    case 128064: return with_rows<E, 128, 64>(rows_a_run, f);
    case 192064: return with_rows<E, 192, 64>(rows_a_run, f);
    case 192128: return with_rows<E, 192, 128>(rows_a_run, f);
    default: return with_rows<E, 128, 128>(rows_a_run, f);
  }
}
template <typename F>
auto with_config(int dtype, int dqk, int dv, int rows_a_run, F f) {
  return dtype == CP_DT_BF16 ? with_dims<__nv_bfloat16>(dqk, dv, rows_a_run, f) : with_dims<float>(dqk, dv, rows_a_run, f);
}

struct Layout {
  int rows, row_tiles, rows_a_run, ctas;
  int cluster;
  size_t parts, total;
};
// Rows of a run: 16, 32 or 64 (fp32: 32, their queries take twice the room); more take several passes over the cache.
// 8 x 8K, 32/8 heads: 64 rows in one pass 64 us, two of 32 94 us, four of 16 167 us; 20 rows in one of 32 52 us, two of 16 87.
// Few runs of few tiles: a cluster a run, joined in shared memory, one launch and no workspace.
Layout layout_of(int num_seqs, int hq, int hkv, int dqk, int dv, int dtype, int n_q, int64_t most) {
  Layout x;
  x.rows = hq / hkv * n_q;
  x.rows_a_run = x.rows <= 16 ? 16 : x.rows <= 32 || dtype == CP_DT_F32 ? 32 : 64;
  x.row_tiles = (x.rows + x.rows_a_run - 1) / x.rows_a_run;
  x.ctas = 2 * sm_count();
  const int64_t runs = int64_t(num_seqs) * hkv * x.row_tiles;
  x.cluster = 0;
  const bool two = with_config(dtype, dqk, dv, x.rows_a_run, [](auto c) { return Room<decltype(c)>::two; });
  const int at_once = two ? x.ctas : x.ctas / 2;
  if (most <= kClusterTokens)
    for (int n = 8; n >= 4 && x.cluster == 0; n /= 2)
      if (runs * n <= at_once) x.cluster = n;
  x.parts = x.total = 0;
  if (x.cluster) return x;
  x.parts = (size_t(x.ctas) * sizeof(int4) + 255) / 256 * 256;
  x.total = (x.parts + size_t(x.ctas) * 2 * x.rows_a_run * (dv + 4) * 4 + 255) / 256 * 256;
  return x;
}

template <typename C>
cudaError_t launch(const KvAttnArgs& a, const Layout& x, cudaStream_t st) {
  Params p;
  p.a = a;
  p.group = a.c.hq / a.c.hkv;
  p.rows = x.rows;
  p.row_tiles = x.row_tiles;
  p.box_shift = std::min(a.c.page_shift, C::F32 ? 5 : 6);
  p.meta = reinterpret_cast<int4*>(a.ws);
  p.parts = reinterpret_cast<float*>(a.ws + x.parts);
  const int64_t pool_rows = (int64_t(a.c.num_pages) * a.c.hkv) << a.c.page_shift;
  // (a pool without pages is not read: any aligned address will do for its map)
  const void* any = a.q;
  const bool none = pool_rows == 0;
  if (!make_map(&p.tk, none ? any : a.c.k, C::F32, none ? 1 : pool_rows, C::DQK, 1 << p.box_shift) ||
      !make_map(&p.tv, none ? any : a.c.v, C::F32, none ? 1 : pool_rows, C::DV, 1 << p.box_shift))
    return cudaErrorInvalidValue;
  p.cluster = x.cluster;
  auto kernel = kv_attn_kernel<C>;
  static std::atomic<uint64_t> ready{0};  // devices whose kernel may use that much shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    // the warps' shares of the registers wait for each other if they add up to more than the CTA started with
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != kLaunchRegs) return cudaErrorInvalidDeviceFunction;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Room<C>::bytes));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  const int ctas = Room<C>::two ? x.ctas : x.ctas / 2;
  const int64_t runs = int64_t(a.c.num_seqs) * a.c.hkv * x.row_tiles;
  // (an entry a run: a CTA of the second kernel for every CTA of the first takes 1 x 16K from 19.0 to 23.0 us)
  p.by_run = runs <= x.ctas;
  p.join_ctas = ctas;
  cudaLaunchAttribute attr{};
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (x.cluster) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(x.cluster);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(unsigned(runs * x.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Room<C>::bytes;
    return cudaLaunchKernelEx(&cfg, kernel, p);
  }
  kernel<<<unsigned(ctas), kThreads, Room<C>::bytes, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the launch overlaps the kernel before: it waits on the device
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  // warps a row: eight for up to 8 rows, one for 64 (a CTA for every row of every run that might be cut takes 10 us)
  const int rows = std::min(x.rows, x.rows_a_run);
  const int rows_a_cta = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 8;
  cfg.gridDim = dim3(unsigned(p.by_run ? runs : ctas), unsigned((rows + rows_a_cta - 1) / rows_a_cta));
  // 32 warps for few rows where a run's parts are many, as long as all of them are there at once: one run of 64 rows over
  // 32K tokens, in 304 parts, 75 us with eight warps for eight rows, 35 us with 32 for eight, 20 us with 32 for two; but 32
  // runs of 32 rows 35 us with eight for four, 53 us with 32 for one
  if (runs * 12 <= ctas) {
    int few = (rows_a_cta + 3) / 4;
    while (runs * ((rows + few - 1) / few) > ctas) few *= 2;
    if (few <= rows_a_cta) {
      cfg.gridDim.y = unsigned((rows + few - 1) / few);
      cfg.blockDim = dim3(32 * 32);
      return cudaLaunchKernelEx(&cfg, kv_join_kernel<C, 32>, p, few);
    }
  }
  cfg.blockDim = dim3(32 * 8);
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<C, 8>, p, rows_a_cta);
}

Layout layout_of(const cp_kv_t* c, int32_t n_q) {
  return layout_of(c->num_seqs, c->hq, c->hkv, c->d_qk, c->d_v, c->dtype, n_q, int64_t(c->max_pages) * c->page_size);
}

}  // namespace

size_t kv_attn_workspace(const cp_kv_t* c, int32_t n_q) { return layout_of(c, n_q).total; }

int64_t kv_attn_units(const cp_kv_t* c, int32_t n_q) {
  const int64_t tiles = (int64_t(c->max_pages) * c->page_size + 31) / 32 + 1;
  return tiles * c->num_seqs * c->hkv * layout_of(c, n_q).row_tiles;
}

cudaError_t launch_kv_attn(const KvAttnArgs& a, int dqk, int dv, int dtype, cudaStream_t st) {
  const Layout x = layout_of(a.c.num_seqs, a.c.hq, a.c.hkv, dqk, dv, dtype, a.n_q, int64_t(a.c.max_pages) << a.c.page_shift);
  return with_config(dtype, dqk, dv, x.rows_a_run, [&](auto c) { return launch<decltype(c)>(a, x, st); });
}

}  // namespace cpattn
