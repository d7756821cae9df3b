// key_weights_sm103.cu — accumulated attention weight of every key of a
// prompt, on the sm_103a tensor cores (tcgen05 + TMEM + TMA).
//
//   w[c, j] = sum over c's query heads h and the queries i that see key j of
//             exp(scale q_i.k_j - lse_i)
// which is a column sum of the attention probabilities, rebuilt from the
// forward's lse as the backward rebuilds them ("Ulysses与Ring-Attention详解"
// §4.3).  The key-major walk is the dK/dV kernel's: one CTA owns a key
// tile of one kv head and visits, for every query head of the group, the
// query runs that see it.  With S^T = K Q^T a thread holds a whole key row
// (TMEM lane = key), so its column sum is a sum over its own registers: no
// exchange between threads, nothing written but one float a key.
//
// A CTA's key tile has 256 rows, two M = 128 halves, so that a Q tile brought
// in from L2 serves two MMAs.  With 128 rows the copies (32 KB a step of 512
// tensor cycles) ran at some 36 bytes a cycle and SM, and the kernel with them.
// Per 128 x 128 half step the tensor cores need 512 cycles (128-wide heads),
// and as much at 32 exponentials a cycle.  K lives in TMEM (a TS MMA): as an SS
// MMA both operands and the Q copies together asked shared memory for 96 KB a
// step, 768 cycles (16K tokens, 32 heads: 1.64 ms, against 0.98 ms).  S^T has
// three TMEM buffers (two with 192-wide heads), each read by a group of four
// warps that takes its tiles in turn, so that one group's loads and waits overlap the others'
// exponentials (two groups: 1.10 ms; a part of the exponentials as polynomials
// on the FMA pipes instead: 1.09 ms and up, the issue slots are needed
// elsewhere).  As it stands 16K tokens of 32 / 8 heads take 0.89 ms, 1.2
// PFLOP/s over the visible pairs.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "plan_check.cuh"
#include "query_steps.cuh"
#include "sm103_ptx.cuh"

namespace cpattn {

bool make_map_3d(CUtensorMap* map, const void* base, CUtensorMapDataType dt, int elt, int64_t dim, int64_t heads,
                 int64_t T, int box_inner, int box_rows, CUtensorMapSwizzle swz);

namespace {

constexpr int BT = 128;                 // keys of a half tile, queries of a step
constexpr uint32_t kPanel = 128 * 128;  // 128 rows x 64 bf16 columns, 128-byte swizzled: 16 KiB
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kGroupThreads = 128;
constexpr unsigned kPhases = 8;
constexpr int kPieceMaps = 15;  // boxes of 8, 16, ..., 120 rows for the pieces of gathered tiles

enum WaitSite : int { kSiteK = 0x61, kSiteQEmpty, kSiteQFull, kSiteSFull, kSiteSFree, kSiteDrain, kSiteAlign };

struct Params {
  CUtensorMap tq;
  CUtensorMap tqp[kPieceMaps];  // plans with gathered query tiles only
  AttnArgs a;
  int32_t* err;
};

template <int DQK>
struct Cfg {
  static constexpr int kPanels = DQK / 64;
  static constexpr int NS = DQK == 128 ? 6 : 4;     // stages of Q
  static constexpr int kBufs = DQK == 128 ? 3 : 2;  // S^T buffers of 128 TMEM columns; K's halves behind them
  // Compute groups: one a buffer, so that a group waits only for the phase after the one it freed (a barrier's parity
  // tells a phase from the next one only).
  static constexpr int kGroups = kBufs;
  static constexpr int kThreads = kGroups * kGroupThreads + 64;
  static constexpr int kProducer = 4 * kGroups, kIssuer = kProducer + 1;  // warps
  static constexpr uint32_t kTileBytes = kPanels * kPanel;
  static constexpr uint32_t offQ = 0;
  static constexpr uint32_t offStat = offQ + NS * kTileBytes;  // [group][2][BT] floats
  static constexpr uint32_t offBar = offStat + kGroups * 2 * BT * 4;
  static constexpr int kNumBars = 1 + 2 * NS + 2 * kBufs;
  static constexpr uint32_t kSmem = offBar + kNumBars * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory budget");
  static constexpr uint32_t tK = kBufs * BT;  // TMEM column of K (packed bf16 pairs)
  static_assert(tK + DQK <= 512, "TMEM budget");
};

// -lse * log2e of query column `col` of the step the cursor points at, -inf
// where the step holds no query or one that is left out (lse = +inf).
template <bool PACKED>
__device__ __forceinline__ float load_stat(const AttnArgs& a, const StepCursor<BT>& c, int col) {
  int64_t row = -1;
  if (PACKED && c.packed()) {
    const int count = c.cur.flags >> kPackCountShift;
    for (int i = 0; i < count; ++i) {
      const PackPiece pc = a.pieces[c.cur.row0 + i];
      if (col >= pc.dst && col < pc.dst + pc.keys) row = int64_t(pc.src) + (col - pc.dst);
    }
  } else if (col < c.n()) {
    row = c.row() + col;
  }
  return row < 0 ? -INFINITY : -(a.lse_in[int64_t(c.head()) * a.T + row] * kLog2e);
}

__device__ __forceinline__ uint64_t exp2_pair(uint64_t y) {
  float a, b;
  ptx::f32x2_split(y, a, b);
  return ptx::f32x2(ptx::ex2(a), ptx::ex2(b));
}

template <int DQK, bool PACKED>
__global__ void __launch_bounds__(Cfg<DQK>::kThreads, 1) key_weights_kernel(const __grid_constant__ Params p) {
  using C = Cfg<DQK>;
  constexpr int NS = C::NS, kBufs = C::kBufs, kGroups = C::kGroups, kProducer = C::kProducer, kIssuer = C::kIssuer;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const AttnArgs& a = p.a;
  if (sbase & 1023u) {  // the swizzled operand panels need 1024-byte alignment
    if (threadIdx.x == 0 && p.err) atomicCAS(p.err, 0, 0x100 | kSiteAlign);
    return;
  }
  // The tiles (heaviest first) in kPhases parts, inside a part kv heads
  // outermost: the CTAs resident at one time read one head's Q, and the last
  // ones to run are light.
  const unsigned part_tiles = unsigned(a.num_tiles + kPhases - 1) / kPhases, per_part = part_tiles * unsigned(a.hkv);
  const unsigned phase = blockIdx.x / per_part, rest = blockIdx.x - phase * per_part;
  const unsigned here = min(part_tiles, unsigned(a.num_tiles) - phase * part_tiles);  // (the last part may be smaller)
  const int kvh = int(rest / here), tile_idx = int(phase * part_tiles + rest - unsigned(kvh) * here);
  if (a.debug && !debug_plan_ok(a, tile_idx, kvh, kvh, true, p.err, 2 * BT)) return;
  const TileDesc tile = a.tiles[tile_idx];
  const int G = a.hq / a.hkv;
  const int n_steps = tile.work * G, halves = tile.nrows > BT ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const uint32_t bar_k = sbase + C::offBar;
  auto bar_q_full = [&](int s) { return bar_k + 8u * (1 + s); };
  auto bar_q_empty = [&](int s) { return bar_k + 8u * (1 + NS + s); };
  auto bar_s_full = [&](int b) { return bar_k + 8u * (1 + 2 * NS + b); };           // S^T of buffer b computed
  auto bar_s_free = [&](int b) { return bar_k + 8u * (1 + 2 * NS + kBufs + b); };   // and read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::offBar + C::kNumBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::offBar + C::kNumBars * 8 + 4);

  if (threadIdx.x == 0) {
    ptx::mbar_init(bar_k, 4 * halves);
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(bar_q_full(s), 2);
      ptx::mbar_init(bar_q_empty(s), 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      ptx::mbar_init(bar_s_full(b), 1);
      ptx::mbar_init(bar_s_free(b), 4);
    }
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == kIssuer) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  if (warp == kProducer && lane == 0) {
    ptx::prefetch_tmap(&p.tq);
  }
  if (PACKED && warp == kProducer && lane >= 1 && lane <= kPieceMaps) ptx::prefetch_tmap(&p.tqp[lane - 1]);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const ptx::WaitCtx wctx{abort_flag, p.err, kWaitLimitNs};

  if (warp == kProducer) {
    // ------------------------------------------------------------ producers: lanes 0 and 1 split the panels
    if (lane < 2 && n_steps > 0) {
      const uint32_t bytes = uint32_t((C::kPanels + 1 - lane) / 2) * kPanel;  // panels lane, lane + 2, ...
      StepCursor<BT> cur;
      cur.init(a.ranges, tile.range_begin, tile.range_count, G, kvh, a.hkv, a.gqa_interleaved);
      int issued = 0;
      for (int i = 0; i < n_steps; ++i, cur.next()) {
        const int st = i % NS;
        if (i >= NS && !ptx::mbar_wait(bar_q_empty(st), ((i / NS) - 1) & 1, kSiteQEmpty, wctx)) break;
        const int h = cur.head();
        const uint32_t dst = sbase + C::offQ + st * C::kTileBytes;
        ptx::mbar_arrive_expect_tx(bar_q_full(st), bytes);
        if (!PACKED || !cur.packed()) {
          for (int c = lane; c < C::kPanels; c += 2)
            ptx::tma_load_3d(dst + c * kPanel, &p.tq, bar_q_full(st), c * 64, h, cur.row());
        } else {
          // one box per piece; the pieces cover the rows of the step from 8-row (1 KiB) boundaries
          const int count = cur.cur.flags >> kPackCountShift;
          for (int k = 0; k < count; ++k) {
            const PackPiece pc = a.pieces[cur.cur.row0 + k];
            const CUtensorMap* m = pc.rows >= BT ? &p.tq : p.tqp + (max(pc.rows, 8) >> 3) - 1;
            for (int c = lane; c < C::kPanels; c += 2)
              ptx::tma_load_3d(dst + c * kPanel + uint32_t(pc.dst) * 128, m, bar_q_full(st), c * 64, h, pc.src);
          }
        }
        ++issued;
      }
      if (*abort_flag) {
        volatile int no_abort = 0;
        const ptx::WaitCtx drain{&no_abort, nullptr, kWaitLimitNs};
        for (int i = max(0, issued - NS); i < issued; ++i)
          ptx::mbar_wait(bar_q_full(i % NS), (i / NS) & 1, kSiteDrain, drain);
      }
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ MMA issuer (whole warp)
    if (n_steps > 0) {
      constexpr uint32_t idS = ptx::idesc_bf16_f32(BT, BT, false, false);
      bool ok = ptx::mbar_wait_w(bar_k, 0, kSiteK, wctx);
      int j = 0;  // S^T tiles issued
      for (int i = 0; ok && i < n_steps; ++i) {
        const int st = i % NS;
        ok = ptx::mbar_wait_w(bar_q_full(st), (i / NS) & 1, kSiteQFull, wctx);
        for (int half = 0; ok && half < halves; ++half, ++j) {
          const int b = j % kBufs;
          ok = j < kBufs || ptx::mbar_wait_w(bar_s_free(b), ((j / kBufs) - 1) & 1, kSiteSFree, wctx);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t dq = ptx::sdesc_sw128(sbase + C::offQ + st * C::kTileBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < DQK / 16; ++kk)
            ptx::mma_ts_w(tmem + b * BT, tmem + C::tK + half * (DQK / 2) + kk * 8,
                          dq + (((kk >> 2) * kPanel + (kk & 3) * 32) >> 4), idS, kk > 0);
          ptx::mma_commit_w(bar_s_full(b));
        }
        if (ok) ptx::mma_commit_w(bar_q_empty(st));
      }
      if (!ok && j > 0) {  // the MMAs issued so far end before the CTA frees its TMEM
        volatile int no_abort = 0;
        const ptx::WaitCtx drain{&no_abort, nullptr, kWaitLimitNs};
        ptx::mbar_wait_w(bar_s_full((j - 1) % kBufs), ((j - 1) / kBufs) & 1, kSiteDrain, drain);
      }
    }
  } else {
    // ------------------------------------------------------------ column sums
    const int grp = warp >> 2;
    const int t = threadIdx.x & (kGroupThreads - 1);  // key row = TMEM lane; column whose statistic it loads
    const uint32_t tS = tmem + (uint32_t((warp & 3) * 32) << 16);
    float* stat = reinterpret_cast<float*>(smem + C::offStat) + grp * 2 * BT;
    const float sl2 = a.scale * kLog2e;
    const uint64_t sl2x2 = ptx::f32x2(sl2, sl2);
    if (grp < halves && n_steps > 0) {
      // K row -> TMEM (bf16 pairs are the A-operand packing).  Rows past the
      // tile are the following ones, or zeros past the end: not written out.
      const int64_t krow = int64_t(tile.row0) + grp * BT + t;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + (krow * a.hkv + kvh) * DQK);
#pragma unroll
      for (int c = 0; c < DQK / 64; ++c) {
        uint32_t kr[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = krow < a.T ? __ldg(src + 8 * c + i) : make_uint4(0, 0, 0, 0);
          kr[4 * i] = v.x, kr[4 * i + 1] = v.y, kr[4 * i + 2] = v.z, kr[4 * i + 3] = v.w;
        }
        ptx::tmem_st32(tS + C::tK + grp * (DQK / 2) + 32 * c, kr);
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar_k);
    }
    StepCursor<BT> cur;
    cur.init(a.ranges, tile.range_begin, tile.range_count, G, kvh, a.hkv, a.gqa_interleaved);
    // group g takes S^T tiles g, g + kGroups, ...: half j % halves of step j / halves
    const int n_tiles = n_steps * halves;
    int step = 0;
    auto go_to = [&](int j) {
      for (const int to = j / halves; step < to; ++step) cur.next();
    };
    float next = 0.f;
    if (grp < n_tiles) {
      go_to(grp);
      next = load_stat<PACKED>(a, cur, t);
    }
    float w[2] = {0.f, 0.f};
    bool ok = true;
    for (int j = grp, k = 0; j < n_tiles; j += kGroups, ++k) {
      const int nq = cur.n(), qpos0 = cur.pos(), b = j % kBufs, half = j % halves;
      const bool packed = PACKED && cur.packed();
      float* st = stat + (k & 1) * BT;
      // (the buffer was last read two of this group's tiles ago, before the barrier of the tile between)
      st[t] = next;
      // (a query left out may hold what it likes: the step is masked)
      const bool left_out = ptx::named_barrier_any(1 + grp, kGroupThreads, next == -INFINITY);
      if (j + kGroups < n_tiles) {
        go_to(j + kGroups);
        next = load_stat<PACKED>(a, cur, t);
      }
      if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait_poll(bar_s_full(b), (j / kBufs) & 1, kSiteSFull, wctx));
      if (!ok) continue;  // keep to the group's barriers
      ptx::tc_fence_after();
      const bool causal = a.causal && !packed;
      const int first = tile.pos0 + half * BT;
      // columns from cmin on are visible; columns without a query, and of one left out, have the statistic -inf
      const bool need_mask = left_out || (causal && qpos0 < first + BT - 1);
      const int cmin = causal ? first + t - qpos0 : 0;
      uint64_t s0 = 0, s1 = 0;  // a step's own sums: a long sum's roundings stay small
      auto sums = [&](auto mask_) {
        constexpr bool MASK = decltype(mask_)::value;
        uint32_t x[2][32];  // 32 columns at hand, the next 32 on their way
        ptx::tmem_ld32(tS + b * BT, x[0]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          ptx::tmem_ld_wait();
          ptx::reg_fence32(x[q & 1]);
          if (q < 3) {
            ptx::tmem_ld32(tS + b * BT + 32 * (q + 1), x[(q + 1) & 1]);
          } else {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_s_free(b));
          }
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const int col = 32 * q + j;
            const float4 nl = *reinterpret_cast<const float4*>(st + col);
            const uint32_t* xs = &x[q & 1][j];
            const uint64_t y0 = ptx::fma_f32x2(ptx::f32x2(__uint_as_float(xs[0]), __uint_as_float(xs[1])), sl2x2,
                                               ptx::f32x2(nl.x, nl.y));
            const uint64_t y1 = ptx::fma_f32x2(ptx::f32x2(__uint_as_float(xs[2]), __uint_as_float(xs[3])), sl2x2,
                                               ptx::f32x2(nl.z, nl.w));
            uint64_t e0 = exp2_pair(y0);
            uint64_t e1 = exp2_pair(y1);
            if (MASK) {
              float v[4];
              ptx::f32x2_split(e0, v[0], v[1]);
              ptx::f32x2_split(e1, v[2], v[3]);
              const float n4[4] = {nl.x, nl.y, nl.z, nl.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (col + e < cmin || n4[e] == -INFINITY) v[e] = 0.f;
              e0 = ptx::f32x2(v[0], v[1]);
              e1 = ptx::f32x2(v[2], v[3]);
            }
            s0 = ptx::add_f32x2(s0, e0);
            s1 = ptx::add_f32x2(s1, e1);
          }
        }
      };
      // warp-uniform: only steps on the diagonal or with columns that do not count pay for the tests
      if (need_mask) sums(std::true_type{});
      else sums(std::false_type{});
      float a0, a1;
      ptx::f32x2_split(ptx::add_f32x2(s0, s1), a0, a1);
      if (half) w[1] += a0 + a1;
      else w[0] += a0 + a1;
    }
    // the groups' sums through shared memory, in their statistics' places once all of a group's threads have read them
    ptx::named_barrier(1 + grp, kGroupThreads);
    stat[t] = w[0];
    stat[BT + t] = w[1];
    ptx::named_barrier(1 + kGroups, kGroups * kGroupThreads);
    if (grp < halves && grp * BT + t < tile.nrows) {
      const float* all = reinterpret_cast<const float*>(smem + C::offStat) + grp * BT + t;
      float sum = all[0];
#pragma unroll
      for (int g = 1; g < kGroups; ++g) sum += all[g * 2 * BT];
      static_cast<float*>(a.out)[int64_t(kvh) * a.T + tile.row0 + grp * BT + t] = sum;
    }
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int DQK>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  using C = Cfg<DQK>;
  Params p;
  p.a = a;
  p.err = device_error_word();
  if (!make_map_3d(&p.tq, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, DQK, a.hq, a.T, 64, BT, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (a.num_packs > 0)
    for (int m = 0; m < kPieceMaps; ++m)
      if (!make_map_3d(&p.tqp[m], a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, DQK, a.hq, a.T, 64, 8 * (m + 1),
                       CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
  auto kernel = a.num_packs > 0 ? key_weights_kernel<DQK, true> : key_weights_kernel<DQK, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem));
  if (e != cudaSuccess) return e;
  const int64_t grid = int64_t(a.num_tiles) * a.hkv;
  if (grid == 0) return cudaSuccess;
  kernel<<<unsigned(grid), C::kThreads, C::kSmem, st>>>(p);
  return cudaGetLastError();
}

// ===========================================================================
// Few queries: the last ones of a prompt (an observation window)
// ===========================================================================
// With G * queries <= 256 all of a kv head's columns are one B operand: it is
// gathered into shared memory once and stays, and the key tiles stream past it
// (the key-major kernel above would start a CTA for every key tile to visit a
// few steps).  The keys are read once and nothing else is: 64K tokens, 8 kv
// heads of 128 are 134 MB, 20 us of HBM; per tile of 128 keys that is 1400
// cycles an SM, the MMA (N = 256) and the exponentials take 1024 each.
// Persistent: the (kv head, key tile) items are cut evenly over the SMs, in
// order, so a CTA gathers queries once or twice.  S has two TMEM buffers, each
// read by eight compute warps, four a half of the columns (with four warps a
// buffer a tile took 4500 cycles: too few warps to hide their latencies).  The
// case above takes 41 us, 3.3 TB/s.

constexpr int kWinCols = 256;
constexpr int kWinThreads = 4 * kGroupThreads + 64;
constexpr int kWinProducer = 16, kWinIssuer = 17;  // warps

struct WinParams {
  CUtensorMap tk;
  AttnArgs a;
  const WinTile* tiles;
  const WinSeq* seqs;
  const int32_t* rows;  // sharded rows of the counted queries
  int32_t num_tiles;
  int32_t* err;
};

template <int DQK>
struct WinCfg {
  static constexpr int kPanels = DQK / 64;
  static constexpr int NS = DQK == 128 ? 4 : 2;  // stages of K
  static constexpr uint32_t kTileBytes = kPanels * kPanel;
  static constexpr uint32_t kQPanel = kWinCols * 128;  // kWinCols rows x 64 bf16 columns
  static constexpr uint32_t offQ = 0;
  static constexpr uint32_t offK = kPanels * kQPanel;
  static constexpr uint32_t offStat = offK + NS * kTileBytes;  // -lse log2e of every column
  static constexpr uint32_t offPos = offStat + kWinCols * 4;   // and its query's position
  static constexpr uint32_t offPart = offPos + kWinCols * 4;   // [parity][2][BT]: sums of the second half's columns
  static constexpr uint32_t offBar = offPart + 4 * BT * 4;
  static constexpr int kNumBars = 2 * NS + 4;
  static constexpr uint32_t kSmem = offBar + kNumBars * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory budget");
};

template <int DQK>
__global__ void __launch_bounds__(kWinThreads, 1) key_weights_window_kernel(const __grid_constant__ WinParams p) {
  using C = WinCfg<DQK>;
  constexpr int NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const AttnArgs& a = p.a;
  if (sbase & 1023u) {
    if (threadIdx.x == 0 && p.err) atomicCAS(p.err, 0, 0x100 | kSiteAlign);
    return;
  }
  const int64_t items = int64_t(a.hkv) * p.num_tiles;
  const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
  if (i0 == i1) return;
  const int G = a.hq / a.hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar_full = [&](int s) { return sbase + C::offBar + 8u * s; };
  auto bar_empty = [&](int s) { return sbase + C::offBar + 8u * (NS + s); };
  auto bar_s_full = [&](int b) { return sbase + C::offBar + 8u * (2 * NS + b); };
  auto bar_s_free = [&](int b) { return sbase + C::offBar + 8u * (2 * NS + 2 + b); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::offBar + C::kNumBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::offBar + C::kNumBars * 8 + 4);
  float* stat = reinterpret_cast<float*>(smem + C::offStat);
  int32_t* qpos = reinterpret_cast<int32_t*>(smem + C::offPos);
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(bar_full(s), 2);
      ptx::mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bar_s_full(b), 1);
      ptx::mbar_init(bar_s_free(b), 8);
    }
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == kWinIssuer) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  if (warp == kWinProducer && lane == 0) ptx::prefetch_tmap(&p.tk);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const ptx::WaitCtx wctx{abort_flag, p.err, kWaitLimitNs};
  const uint64_t sl2x2 = ptx::f32x2(a.scale * kLog2e, a.scale * kLog2e);
  bool ok = true;

  for (int64_t seg = i0; seg < i1;) {
    // ---- a kv head and a sequence: its counted queries become the B operand
    const int kvh = int(seg / p.num_tiles);
    const WinSeq q = p.seqs[p.tiles[seg - int64_t(kvh) * p.num_tiles].seq];
    const int64_t end = min(i1, int64_t(kvh) * p.num_tiles + q.tile0 + q.tiles);
    const int cols = G * q.count, N = (cols + 15) & ~15;
    for (int e = threadIdx.x; e < N * (DQK / 8); e += kWinThreads) {
      const int n = e / (DQK / 8), chunk = e - n * (DQK / 8), g = n / q.count;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (n < cols) {
        const int h = a.gqa_interleaved ? g * a.hkv + kvh : kvh * G + g;
        v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                 (int64_t(p.rows[q.row0 + n - g * q.count]) * a.hq + h) * DQK) + chunk);
      }
      *reinterpret_cast<uint4*>(smem + C::offQ + (chunk >> 3) * C::kQPanel + n * 128 + (((chunk & 7) ^ (n & 7)) << 4)) = v;
    }
    bool out = false;  // columns that do not count: no query, or one left out (lse = +inf)
    for (int n = threadIdx.x; n < kWinCols; n += kWinThreads) {
      const int g = n / q.count, j = n - g * q.count;
      const int h = a.gqa_interleaved ? g * a.hkv + kvh : kvh * G + g;
      stat[n] = n < cols ? -(a.lse_in[int64_t(h) * a.T + p.rows[q.row0 + j]] * kLog2e) : -INFINITY;
      qpos[n] = a.causal ? q.pos0 + j : INT32_MAX;
      out |= stat[n] == -INFINITY && n < ((cols + 31) & ~31);
    }
    ptx::fence_proxy_async_smem();
    const bool left_out = __syncthreads_or(out);

    if (warp == kWinProducer) {
      // ---------------------------------------------------------- producers: lanes 0 and 1 split the panels
      if (lane < 2) {
        const uint32_t bytes = uint32_t((C::kPanels + 1 - lane) / 2) * kPanel;
        for (int64_t i = seg; ok && i < end; ++i) {
          const int64_t k = i - i0;
          const int st = int(k % NS);
          if (k >= NS) ok = ptx::mbar_wait(bar_empty(st), uint32_t((k / NS) - 1) & 1, kSiteQEmpty, wctx);
          if (!ok) break;
          const WinTile t = p.tiles[i - int64_t(kvh) * p.num_tiles];
          ptx::mbar_arrive_expect_tx(bar_full(st), bytes);
          for (int c = lane; c < C::kPanels; c += 2)
            ptx::tma_load_3d(sbase + C::offK + st * C::kTileBytes + c * kPanel, &p.tk, bar_full(st), c * 64, kvh, t.row0);
        }
      }
      __syncwarp();
    } else if (warp == kWinIssuer) {
      // ---------------------------------------------------------- MMA issuer (whole warp)
      const uint32_t idS = ptx::idesc_bf16_f32(BT, 16, false, false) - (2u << 17) + (uint32_t(N >> 3) << 17);
      for (int64_t i = seg; ok && i < end; ++i) {
        const int64_t k = i - i0;
        const int st = int(k % NS), b = int(k & 1);
        ok = ptx::mbar_wait_w(bar_full(st), uint32_t(k / NS) & 1, kSiteQFull, wctx) &&
             (k < 2 || ptx::mbar_wait_w(bar_s_free(b), uint32_t((k >> 1) - 1) & 1, kSiteSFree, wctx));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t dk = ptx::sdesc_sw128(sbase + C::offK + st * C::kTileBytes, 16, 1024);
        const uint64_t dq = ptx::sdesc_sw128(sbase + C::offQ, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < DQK / 16; ++kk)
          ptx::mma_ss_w(tmem + b * kWinCols, dk + (((kk >> 2) * kPanel + (kk & 3) * 32) >> 4),
                        dq + (((kk >> 2) * C::kQPanel + (kk & 3) * 32) >> 4), idS, kk > 0);
        ptx::mma_commit_w(bar_s_full(b));
        ptx::mma_commit_w(bar_empty(st));
      }
    } else {
      // ---------------------------------------------------------- column sums: groups of parity 0 and 1, two halves each
      const int par = warp >> 3, half = (warp >> 2) & 1, t = threadIdx.x & (kGroupThreads - 1);
      const uint32_t tS = tmem + (uint32_t((warp & 3) * 32) << 16) + par * kWinCols;
      float* part = reinterpret_cast<float*>(smem + C::offPart) + par * 2 * BT;
      const int chunks = (N + 31) / 32, ch0 = half ? (chunks + 1) / 2 : 0, ch1 = half ? chunks : (chunks + 1) / 2;
      for (int64_t i = seg + (((seg - i0) & 1) != par); i < end; i += 2) {
        const int64_t k = i - i0;
        const WinTile tile = p.tiles[i - int64_t(kvh) * p.num_tiles];
        const int kpos = tile.pos0 + t * tile.stride;
        const bool need_mask = a.causal && tile.pos0 + (tile.nrows - 1) * tile.stride > q.pos0;
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait_poll(bar_s_full(par), uint32_t(k >> 1) & 1, kSiteSFull, wctx));
        float w = 0.f;
        if (ok) {
          ptx::tc_fence_after();
          auto sums = [&](auto mask_) {
            constexpr bool MASK = decltype(mask_)::value;
#pragma unroll 1
            for (int ch = ch0; ch < ch1; ++ch) {  // 32 columns
              uint32_t x[32];
              ptx::tmem_ld32(tS + 32 * ch, x);
              ptx::tmem_ld_wait();
              ptx::reg_fence32(x);
              uint64_t s0 = 0, s1 = 0;
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 nl = *reinterpret_cast<const float4*>(stat + 32 * ch + j);
                uint64_t e0 = exp2_pair(ptx::fma_f32x2(ptx::f32x2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), sl2x2,
                                                       ptx::f32x2(nl.x, nl.y)));
                uint64_t e1 = exp2_pair(ptx::fma_f32x2(ptx::f32x2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])),
                                                       sl2x2, ptx::f32x2(nl.z, nl.w)));
                if (MASK) {
                  float v[4];
                  ptx::f32x2_split(e0, v[0], v[1]);
                  ptx::f32x2_split(e1, v[2], v[3]);
                  const float n4[4] = {nl.x, nl.y, nl.z, nl.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (kpos > qpos[32 * ch + j + e] || n4[e] == -INFINITY) v[e] = 0.f;
                  e0 = ptx::f32x2(v[0], v[1]);
                  e1 = ptx::f32x2(v[2], v[3]);
                }
                s0 = ptx::add_f32x2(s0, e0);
                s1 = ptx::add_f32x2(s1, e1);
              }
              float a0, a1;
              ptx::f32x2_split(ptx::add_f32x2(s0, s1), a0, a1);
              w += a0 + a1;
            }
          };
          // (columns from cols on are products with zeros, NaN where a key is infinite, and from N on stale: masked too,
          // like those of a query left out, which may hold what it likes)
          if (need_mask || left_out) sums(std::true_type{});
          else sums(std::false_type{});
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar_s_free(par));
        }
        // the halves meet; the place is used again two of this parity's items on, past the barrier between
        float* p2 = part + (uint32_t(k >> 1) & 1) * BT;
        if (half) p2[t] = w;
        ptx::named_barrier(1 + par, 2 * kGroupThreads);
        if (!half && t < tile.nrows)
          static_cast<float*>(a.out)[int64_t(kvh) * a.T + tile.row0 + t] = w + p2[t];
      }
    }
    __syncthreads();  // the operand and the statistics have been read
    seg = end;
  }
  // what was issued ends before the CTA goes: after a wait that gave up, the copies and the MMAs still in flight
  if (*abort_flag && warp == kWinProducer && lane == 0) {
    volatile int no_abort = 0;
    const ptx::WaitCtx drain{&no_abort, nullptr, kWaitLimitNs / 4};
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_wait(bar_full(s), 0, kSiteDrain, drain);
      ptx::mbar_wait(bar_full(s), 1, kSiteDrain, drain);
    }
    for (int b = 0; b < 2; ++b) ptx::mbar_wait(bar_s_full(b), 0, kSiteDrain, drain);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kWinIssuer) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int DQK>
cudaError_t launch_window(const AttnArgs& a, const WinTile* tiles, int32_t num_tiles, const WinSeq* seqs,
                          const int32_t* rows, int sms, cudaStream_t st) {
  using C = WinCfg<DQK>;
  WinParams p;
  p.a = a;
  p.tiles = tiles;
  p.seqs = seqs;
  p.rows = rows;
  p.num_tiles = num_tiles;
  p.err = device_error_word();
  if (!make_map_3d(&p.tk, a.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, DQK, a.hkv, a.T, 64, BT, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(key_weights_window_kernel<DQK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(C::kSmem));
  if (e != cudaSuccess) return e;
  const int64_t items = int64_t(num_tiles) * a.hkv;
  if (items == 0) return cudaSuccess;
  key_weights_window_kernel<DQK><<<unsigned(std::min<int64_t>(items, sms)), kWinThreads, C::kSmem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

bool key_weights_window_supported(int32_t d_qk, int32_t columns) {
  return tc_key_weights_supported(d_qk) && columns <= kWinCols;
}

cudaError_t launch_key_weights_window(const AttnArgs& a, const WinTile* tiles, int32_t num_tiles, const WinSeq* seqs,
                                      const int32_t* rows, int32_t sms, cudaStream_t st) {
  if (a.d_qk == 128) return launch_window<128>(a, tiles, num_tiles, seqs, rows, sms, st);
  if (a.d_qk == 192) return launch_window<192>(a, tiles, num_tiles, seqs, rows, sms, st);
  return cudaErrorInvalidValue;
}

bool tc_key_weights_supported(int32_t d_qk) { return d_qk == 128 || d_qk == 192; }

cudaError_t launch_tc_key_weights(const AttnArgs& a, cudaStream_t st) {
  if (a.d_qk == 128) return launch<128>(a, st);
  if (a.d_qk == 192) return launch<192>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace cpattn
