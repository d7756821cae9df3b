// kv4_attn.cu — attention of single tokens (or a few) over the 4-bit cache.
//
// Row (b, t, h) sees slots j < lengths[b] - (n_q - 1 - t):
//   S_j = scale q.K_j,  lse = log sum_j exp(S_j),  o = sum_j exp(S_j - lse) V_j.
// The cache is read once (144 bytes a token's head of 128 + 128 channels), and
// every byte meets G * n_q rows.  At 6.7 TB/s an SM gets about 23 bytes a
// cycle, 46 codes; unpacking them, the MMAs' operands and the scales take more
// issue slots than that leaves, so the long cases are bound by instruction
// issue (8 x up to 64K tokens, d 128: 77 us, 59% of issue slots, ALU pipe 53%,
// 44% of the measured copy rate; 128K tokens, 64 heads, d 192/128: 348 us,
// 64% and 64%), the short ones by latency (16K tokens: 15 us, and 7 to join).
//
// Warp-level MMAs, not tcgen05: with 1 to 16 rows a tcgen05 tile would be
// nearly empty, and its operands would have to be unpacked into shared or
// tensor memory first; here a lane's packed words are unpacked in registers
// straight into the fragments (keys or channels on the 16 side, rows on the 8
// side), which the format's word order was chosen for.
//
// * K of bf16 caches: a code's nibble in a byte is the e4m3 number n 2^-9, so
//   one AND (and a shift) makes four operands of mma.m16n8k32.  A query row is
//   scaled by a power of two to a largest channel of 128 .. 256 and split into
//   two e4m3 terms: 8 bits, all that bf16 has.  Each product starts from zero
//   and is added to S by FMAs with the group's scale.  (bf16 operands would
//   take as many MMAs, one term over twice the steps, but an instruction more
//   for every two codes to unpack.)
// * V, and K of fp32 caches: a code becomes the bf16 number n - 8 (below) for
//   mma.m16n8k16.  fp32 caches split q and P s into three bf16 terms (24 bits).
// * Scales and lows act in fp32: on S per (key, group), the lows on sum(q); on
//   P per (token, group), the lows (with 8 steps added) on a sum of their own.
// * P s of a bf16 cache is rounded to one bf16 operand, as P is in the prompt's
//   forward; the softmax sum takes it unrounded.  O is then 0.0019 to 0.0024 of
//   its norm off (fp32 arithmetic rounded to bf16 once: 0.0016), in fp32
//   partials too.  A second term would double V's MMAs; who needs more opens
//   the same pages in a descriptor of dtype FP32 (three terms: 2e-7).
// * S^T comes out with keys as rows and goes back in as P^T with tokens as
//   the contracted index: movmatrix transposes the 8 x 8 quarters.
// * The softmax keeps a reference per row instead of a running maximum: P =
//   2^(S - ref), and only when an element exceeds the reference by more than
//   2^10 does the warp take a new maximum and rescale.
//
// Work: every (sequence, kv head, row tile) is a run of units, one for its
// start (the queries are made operands) and one a sub-block of 32 tokens; all
// runs laid end to end are cut evenly over the CTAs (one an SM) and their
// warps, whatever the lengths, on the device: a graph replays with other
// lengths.  A warp has a ring of copies of its own and waits for nobody.
// 12 warps (10, 14 and 16 were slower: registers against latency), 8 where two
// row tiles or three terms need the registers.  What a warp leaves of a run
// that goes on elsewhere is joined in the CTA first; runs that lie in one CTA
// are finished there, the others leave partials for kv4_join_kernel.  Weights
// need the final lse: the scores, 4 bytes a row and slot, wait in the workspace
// (in L2 as far as they fit: 4 x 64K of 16 / 4 heads are 17 MB, 8 x 64K of 32 / 8
// with 4 queries 268 MB) and kv4_weights_kernel adds them up.  Both are launched while the kernel before
// them drains.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include <cuda_fp8.h>

#include "kv4.cuh"
#include "sm103_ptx.cuh"

namespace cpattn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoRef = -1e30f;   // a row that has seen nothing
constexpr float kSlack = 10.f;     // how far (log2) an element may exceed the reference

template <int DQK_, int DV_, int NT_, int TERMS_, int NW_>
struct Cfg {
  static constexpr int DQK = DQK_, DV = DV_, NT = NT_, TERMS = TERMS_, NW = NW_;
  static constexpr int GK = DQK / 64, GV = DV / 64;
  static constexpr int KW = DQK / 32;  // words of a K row a lane unpacks
  static constexpr int COLS = 8 * NT;
  static constexpr int THREADS = 32 * NW;
  static constexpr int SUB = Kv4Format(DQK, DV).sub();
  static constexpr int STAGES = SUB <= 2400 ? 4 : (SUB <= 3500 ? 3 : 2);  // sub-blocks on their way to a warp
};

// The shares: all runs end to end, a run being one unit for its start (its
// queries are made operands, which takes about as long as a sub-block) and
// one a sub-block, cut over n CTAs; a unit a warp at least (a CTA with fewer
// takes as long, and every CTA that a run is cut over leaves a partial to
// join).  No share is empty.
__device__ __forceinline__ int share_count(int units, int ctas, int warps) { return min(ctas, (units + warps - 1) / warps); }
__host__ __device__ __forceinline__ int64_t share_begin(int64_t units, int n, int c) { return int64_t(c) * units / n; }
__device__ __forceinline__ int share_of(int64_t units, int n, int64_t u) { return int(((u + 1) * n - 1) / units); }

// Partial result of a run in a CTA's share: [m][l] of COLS rows, then o.
__host__ __device__ constexpr int part_floats(int cols, int dv) { return 2 * cols + cols * dv; }

struct Grid {
  int ctas;           // shares at most
  int warps;          // of a CTA of the first kernel
  int rows_per_tile;  // rows of a row tile (at most COLS)
  uint32_t off_base, off_frag, off_stat, off_stash, off_ring;
  uint32_t off_join;  // the join's weights behind its scan
  float* part;   // [ctas][2][part_floats]
  float* score;  // [units][rows_per_tile][32], log2 units
};

// First unit of every sequence (base[b], base[num_seqs] = all): the CTA's
// threads fill it.  per: runs a sequence has (hkv * row tiles).
template <int THREADS>
__device__ void scan_lengths(const Kv4AttnArgs& a, int per, int32_t* base, int32_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int carry = 0;
  for (int b0 = 0; b0 < a.c.num_seqs; b0 += THREADS) {
    const int b = b0 + tid;
    const int subs = b < a.c.num_seqs ? (kv4_length(a.c, a.lengths, b) + kKv4Sub - 1) / kKv4Sub : 0;
    int x = subs > 0 ? (subs + 1) * per : 0;
    const int own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int before = carry, all = carry;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += scratch[w];
      all += scratch[w];
    }
    if (b < a.c.num_seqs) base[b] = before + x - own;
    carry = all;
    __syncthreads();
  }
  if (tid == 0) base[a.c.num_seqs] = carry;
  __syncthreads();
}

// The sequence that holds unit u, searched from b on (base[b] <= u < base[num_seqs]).
__device__ __forceinline__ int seq_of_unit(const int32_t* base, int n, int b, int u) {
  if (u < base[b + 1]) return b;
  int lo = b + 1, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (u < base[mid + 1]) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Masks of the unpacking in registers (a LOP3 has room for one immediate, and
// the compiler, seeing two, makes two instructions of each).
struct Masks {
  uint32_t nib, sixteen, low, big;
  __device__ Masks() {
    asm("mov.u32 %0, 0x00780078;" : "=r"(nib));
    asm("mov.u32 %0, 0x41804180;" : "=r"(sixteen));
    asm("mov.u32 %0, 0x000f000f;" : "=r"(low));
    asm("mov.u32 %0, 0x43004300;" : "=r"(big));
  }
};
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t a, uint32_t o) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(a), "r"(o));
  return y;
}
// n - 8 of nibbles I and I + 4 as a bf16 pair, exact: 16 + n is put together from bits and 24 taken off. Around the
// middle, because sums over many tokens cancel: with 16 + n or 0 + n the fp32 accumulators (which the tensor cores cut
// off rather than round) carry 8 to 24 times the sum of P s, and the rounding of P s to bf16 is worth up to 15 steps
// instead of 8. (128K tokens, d 192/128: error of O 0.047 of its norm with 16 + n.)
template <int I>
__device__ __forceinline__ uint32_t nibbles(uint32_t w, const Masks& k) {
  return ptx::add_bf16x2(and_or(I == 0 ? w << 3 : w >> (4 * I - 3), k.nib, k.sixteen), 0xC1C0C1C0u);
}

// Nibbles 0 and 4, by way of 128 + n, which takes no shift
__device__ __forceinline__ uint32_t nibble0(uint32_t w, const Masks& k) {
  return ptx::add_bf16x2(and_or(w, k.low, k.big), 0xC308C308u);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// bf16 number i of packed words
template <int N>
__device__ __forceinline__ float half_at(const uint32_t (&w)[N], int i) {
  return (i & 1) ? bf_hi(w[i >> 1]) : bf_lo(w[i >> 1]);
}

// N packed words of shared memory (aligned to the widest load that N allows)
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p + 4 * i);
      w[i] = v.x, w[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
  }
}
__device__ __forceinline__ float load_bf16(const uint8_t* p) {
  return __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(p)) << 16);
}

// x as TERMS bf16 terms, the first the nearest
template <int TERMS>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&t)[TERMS]) {
#pragma unroll
  for (int i = 0; i < TERMS; ++i) {
    t[i] = ptx::pack_bf16(x, y);
    if (i + 1 < TERMS) {
      x -= bf_lo(t[i]);
      y -= bf_hi(t[i]);
    }
  }
}

__device__ __forceinline__ uint32_t e4m3_pair(float x, float y) {  // x in the low byte
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
// x (|x| < 256) as the e4m3 number next to it, and what is left: four significant bits (Dekker's splitting), then a
// multiple of 2^-9, e4m3's smallest step, which what has four bits above 2^-6 is already. Both differences are exact, so
// that the second term makes up for all that the first one's rounding left: off by 2^-10 at most, and only where x has
// bits below 2^-9.
__device__ __forceinline__ void split4(float x, float& high, float& rest) {
  const float t = __fmul_rn(x, 1048577.f);  // 2^20 + 1
  high = __fsub_rn(t, __fsub_rn(t, x));
  high = __fsub_rn(__fadd_rn(high, 24576.f), 24576.f);  // 1.5 2^14: its last bit is 2^-9
  rest = __fsub_rn(x, high);
}

__device__ __forceinline__ void load_q8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load_q8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  x[0] = bf_lo(a.x), x[1] = bf_hi(a.x), x[2] = bf_lo(a.y), x[3] = bf_hi(a.y);
  x[4] = bf_lo(a.z), x[5] = bf_hi(a.z), x[6] = bf_lo(a.w), x[7] = bf_hi(a.w);
}

__device__ __forceinline__ void store_o4(const Kv4AttnArgs& a, int64_t i, float4 x) {
  if (a.o_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.o) + i) = x;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + i) =
        make_uint2(ptx::pack_bf16(x.x, x.y), ptx::pack_bf16(x.z, x.w));
}
__device__ __forceinline__ void store_o(const Kv4AttnArgs& a, int64_t i, float x) {
  if (a.o_f32) static_cast<float*>(a.o)[i] = x;
  else static_cast<__nv_bfloat16*>(a.o)[i] = __float2bfloat16_rn(x);
}

// Row n of a row tile of kv head h of sequence b: its (b, t, head) row of q and o, and t
__device__ __forceinline__ int64_t row_index(const Kv4AttnArgs& a, int b, int h, int n, int* t, int* head) {
  const int G = a.c.hq / a.c.hkv;
  *t = n / G;
  const int g = n - *t * G;
  *head = a.c.inter ? g * a.c.hkv + h : h * G + g;
  return (int64_t(b) * a.n_q + *t) * a.c.hq + *head;
}

// Walks units: unit i of run `run` of sequence b, its start (i = 0) or sub-block i - 1.
struct UnitCursor {
  int b, run, i, per_run, h;  // h: the run's kv head
  __device__ void seek(const int32_t* base, int n, int per, int row_tiles, int u) {
    b = seq_of_unit(base, n, 0, u);
    per_run = (base[b + 1] - base[b]) / per;
    run = (u - base[b]) / per_run;
    i = u - base[b] - run * per_run;
    h = run / row_tiles;
  }
  __device__ void next(const int32_t* base, int n, int per, int row_tiles) {
    if (++i < per_run) return;
    i = 0;
    h = ++run / row_tiles;
    if (run < per) return;
    run = h = 0;
    do ++b;
    while (b < n && base[b + 1] == base[b]);
    per_run = b < n ? (base[b + 1] - base[b]) / per : 1;
  }
};

template <typename C, typename E>
__global__ void __launch_bounds__(C::THREADS, 1) kv4_attn_kernel(const Kv4AttnArgs a, const Grid gr) {
  constexpr int NT = C::NT, GK = C::GK, GV = C::GV, NW = C::NW, DQK = C::DQK, DV = C::DV, TERMS = C::TERMS, STAGES = C::STAGES;
  constexpr Kv4Format f(DQK, DV);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t s_scan[NW];
  // partials of runs cut over warps: the run of warp w's first (slot 2w) and of its last (2w + 1), or -1; then the slots
  // that hold one, in order, and where in that list a run's begin
  __shared__ int32_t s_run[2 * NW], s_slot[2 * NW], s_group[2 * NW + 1], s_groups;
  int32_t* base = reinterpret_cast<int32_t*>(smem + gr.off_base);
  float* stat_s = reinterpret_cast<float*>(smem + gr.off_stat);    // [2 NW][2][COLS]: the partials' references and sums
  float* top_s = stat_s + 2 * NW * 2 * C::COLS;                    // [2 NW][COLS]: the largest of a run's references
  float* stash_s = reinterpret_cast<float*>(smem + gr.off_stash);  // [NW][rows_per_tile][DV]: the first partials
  float* last_s = reinterpret_cast<float*>(smem + gr.off_ring);    // the last ones, once no warp uses its ring
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int row_tiles = a.row_tiles, per = a.c.hkv * row_tiles;
  const uint8_t* ring_p = smem + gr.off_ring + warp * (STAGES * f.sub());
  const uint32_t ring = ptx::smem_u32(ring_p);
  if (lane == 0) s_run[2 * warp] = s_run[2 * warp + 1] = -1;
  scan_lengths<C::THREADS>(a, per, base, s_scan);
  const int units = base[a.c.num_seqs];
  const int shares = share_count(units, gr.ctas, NW);
  if (int(blockIdx.x) >= shares) return;
  const int u0 = int(share_begin(units, shares, blockIdx.x)), u1 = int(share_begin(units, shares, blockIdx.x + 1));
  // this warp's units
  const int w0 = u0 + (u1 - u0) * warp / NW, w1 = u0 + (u1 - u0) * (warp + 1) / NW;

  // ---- its copies, STAGES ahead, 16 bytes a lane at a time
  UnitCursor cur, ahead;
  int load_unit = w0, load_stage = 0;
  uint32_t absent = 0;  // bit s: the page of stage s's sub-block is not in the pool
  int next_page = 0;
  auto look_up = [&]() {  // the next sub-block, past starts of runs
    if (load_unit < w1 && ahead.i == 0) {
      ++load_unit;
      ahead.next(base, a.c.num_seqs, per, row_tiles);
    }
    if (load_unit < w1)
      next_page = __ldg(a.c.table + int64_t(ahead.b) * a.c.max_pages + (ahead.i - 1) / (CP_KV4_PAGE / kKv4Sub));
  };
  auto load_next = [&]() {
    if (load_unit < w1) {
      // looked up a unit ago; judged only now, so that nothing waited for it
      const int page = next_page < a.c.num_pages ? next_page : -1;
      if (page >= 0) {
        const uint8_t* src = a.c.pages + (int64_t(page) * a.c.hkv + ahead.h) * f.block() +
                             (ahead.i - 1) % (CP_KV4_PAGE / kKv4Sub) * f.sub() + lane * 16;
        const uint32_t dst = ring + load_stage * f.sub() + lane * 16;
#pragma unroll
        for (int o = 0; o < f.sub(); o += 512)
          if (o + 512 <= f.sub() || lane * 16 < f.sub() - o) ptx::cp_async16(dst + o, src + o);
        absent &= ~(1u << load_stage);
      } else {
        kv4_error(a.c, kKv4Page);
        absent |= 1u << load_stage;
      }
      if (++load_stage == STAGES) load_stage = 0;
      ++load_unit;
      ahead.next(base, a.c.num_seqs, per, row_tiles);
      look_up();
    }
    ptx::cp_async_commit();  // a group a call, empty or not: the waits count them
  };
  if (w0 < w1) {
    cur.seek(base, a.c.num_seqs, per, row_tiles, w0);
    ahead = cur;
    {  // the first run's queries on their way too
      int t, head;
      const int n = (cur.run - cur.h * row_tiles) * gr.rows_per_tile + r % gr.rows_per_tile;
      const E* q = static_cast<const E*>(a.q) + row_index(a, cur.b, cur.h, min(n, a.rows - 1), &t, &head) * DQK;
      for (int o = c * 32; o < DQK * int(sizeof(E)); o += 128)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<const char*>(q) + o));
    }
    look_up();
#pragma unroll
    for (int s = 0; s < STAGES; ++s) load_next();
  }
  ptx::grid_launch_dependents();

  constexpr int kFragStride = C::COLS * 32;
  uint8_t* frag0 = smem + gr.off_frag + warp * (DQK / 16 * TERMS) * kFragStride;
  float O[GV][4][NT][4], ref[NT][2];
  uint64_t ooff2[GV][NT], sum2[NT];  // pairs: columns 2c and 2c + 1
  const Masks masks;
  int stage = 0;
  bool last = false;  // last: the registers hold a partial that the next warp's units continue
  for (int u = w0; u < w1 && !last;) {
    // ---- a run, as far as this warp's units go
    const int b = cur.b, run = cur.run, h = cur.h, run0 = u - cur.i, per_run = cur.per_run;
    const int seg1 = min(w1, run0 + per_run), real0 = run0 + 1;  // sub-blocks from unit real0 on
    if (cur.i == 0) {
      ++u;
      cur.next(base, a.c.num_seqs, per, row_tiles);
      if (u >= w1) break;  // the next warp has all of its sub-blocks
    }
    const int n0 = (run - h * row_tiles) * gr.rows_per_tile;
    const int rows = min(gr.rows_per_tile, a.rows - n0);
    const int len = min(kv4_length(a.c, a.lengths, b), (per_run - 1) * kKv4Sub);
    // ---- its queries as B fragments (kstep 2j + p: channels 8w + 2p, 8w + 2p + 4 and the next two, w = 4j + c), and
    // the sums of their groups.  Columns past the rows repeat rows; nothing of them is written out.
    uint64_t qsum2[GK][NT];
    float sl2[NT][2];
    int lim[NT][2];
    uint8_t* frag[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = (nt * 8 + r) % rows;
      frag[nt] = frag0 + (n * 4 + c) * 8;
      int t, head;
      const E* q = static_cast<const E*>(a.q) + row_index(a, b, h, n0 + n, &t, &head) * DQK + 8 * c;
      float gs[GK], x[DQK / 32][8];
#pragma unroll
      for (int j = 0; j < DQK / 32; ++j) {
        load_q8(q + 32 * j, x[j]);
        if (j % 2 == 0) gs[j / 2] = 0.f;
        gs[j / 2] += ((x[j][0] + x[j][1]) + (x[j][2] + x[j][3])) + ((x[j][4] + x[j][5]) + (x[j][6] + x[j][7]));
      }
      float unit = 1.f, factor = a.c.scale * kLog2e;
      if constexpr (TERMS == 1) {
        // the row times a power of two that brings its largest channel to 128 .. 256
        uint32_t big = 0;
#pragma unroll
        for (int j = 0; j < DQK / 32; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) big = max(big, __float_as_uint(x[j][i]) & 0x7fffffffu);
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const int k = big < 0x00800000u ? 0 : 134 - int(min(big, 0x7f800000u) >> 23);  // 7 - exponent
        unit = __uint_as_float(uint32_t(127 + max(min(k, 126), -126)) << 23);
        // codes are n 2^-9 as e4m3 bytes: scores come out times unit / 512
        // (above 0 and finite, whatever the row holds: an unseen slot's score is -inf times it)
        // (in the order that leaves fp32's range only where the result does)
        factor = fmaxf(unit < 1.f ? factor / unit * 512.f : factor * (512.f / unit), 1e-45f);
        if (big >= 0x7f800000u) {  // a row with a NaN or an infinity: NaN in what every key's score adds up
          factor = 1.f;
          gs[0] = NAN;
        }
#pragma unroll
        for (int j = 0; j < DQK / 32; ++j) {
          float hi[8], lo[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) split4(x[j][i] * unit, hi[i], lo[i]);
          // bytes: channels 8w, 8w + 2, .. and 8w + 1, 8w + 3, ..
          uint8_t* to = frag[nt] + 2 * j * kFragStride;
          *reinterpret_cast<uint2*>(to) = make_uint2(e4m3_pair(hi[0], hi[2]) | e4m3_pair(hi[4], hi[6]) << 16,
                                                     e4m3_pair(hi[1], hi[3]) | e4m3_pair(hi[5], hi[7]) << 16);
          *reinterpret_cast<uint2*>(to + kFragStride) = make_uint2(e4m3_pair(lo[0], lo[2]) | e4m3_pair(lo[4], lo[6]) << 16,
                                                                   e4m3_pair(lo[1], lo[3]) | e4m3_pair(lo[5], lo[7]) << 16);
        }
      } else {
#pragma unroll
        for (int j = 0; j < DQK / 32; ++j) {
          uint32_t f0[2][TERMS], f1[2][TERMS];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            split_pair<TERMS>(x[j][2 * p], x[j][2 * p + 4], f0[p]);
            split_pair<TERMS>(x[j][2 * p + 1], x[j][2 * p + 5], f1[p]);
#pragma unroll
            for (int m = 0; m < TERMS; ++m)
              *reinterpret_cast<uint2*>(frag[nt] + ((2 * j + p) * TERMS + m) * kFragStride) = make_uint2(f0[p][m], f1[p][m]);
          }
        }
      }
#pragma unroll
      for (int g = 0; g < GK; ++g) {
        gs[g] += __shfl_xor_sync(0xffffffffu, gs[g], 1);
        gs[g] += __shfl_xor_sync(0xffffffffu, gs[g], 2);
        if (TERMS == 1) gs[g] *= unit * (1.f / 512.f);
        const float q0 = __shfl_sync(0xffffffffu, gs[g], 2 * c * 4), q1 = __shfl_sync(0xffffffffu, gs[g], (2 * c + 1) * 4);
        qsum2[g][nt] = ptx::f32x2(q0, q1);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) sl2[nt][e] = __shfl_sync(0xffffffffu, factor, (2 * c + e) * 4);
      const int own = len - (a.n_q - 1 - t);
#pragma unroll
      for (int e = 0; e < 2; ++e) lim[nt][e] = __shfl_sync(0xffffffffu, own, (2 * c + e) * 4);
    }
    int t_first, head_;
    row_index(a, b, h, n0, &t_first, &head_);
    const int lim_min = len - (a.n_q - 1 - t_first);
    __syncwarp();

#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int g = 0; g < GV; ++g) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[g][i][nt][e] = 0.f;
        ooff2[g][nt] = 0;
      }
      ref[nt][0] = ref[nt][1] = kNoRef;
      sum2[nt] = 0;
    }

    for (; u < seg1; ++u) {
      const int s = stage;
      ptx::cp_async_wait<STAGES - 1>();
      __syncwarp();
      const uint8_t* st = ring_p + s * f.sub();
      const bool gone = (absent >> s) & 1;
      const int j0 = (u - real0) * kKv4Sub;

      // ---- S^T = K Q^T
      uint64_t S2[2][NT][2];  // pairs of columns: row r, row r + 8
      {
        uint32_t kw[2][2][C::KW], kp[2][2][GK];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t tok = mt * 16 + x * 8 + r;
            load_words<C::KW>(st + f.kc() + tok * (DQK / 2) + c * (C::KW * 4), kw[mt][x]);
            load_words<GK>(st + f.kp() + tok * (GK * 4), kp[mt][x]);
          }
#pragma unroll
        for (int g = 0; g < GK; ++g) {
          uint64_t ks[2][2];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float s1 = half_at(kp[mt][x], g);
              float l1 = half_at(kp[mt][x], GK + g);
              if (TERMS == 3) l1 = fmaf(8.f, s1, l1);
              ks[mt][x] = ptx::f32x2(s1, s1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                S2[mt][nt][x] = g == 0 ? ptx::mul_f32x2(ptx::f32x2(l1, l1), qsum2[0][nt])
                                       : ptx::fma_f32x2(ptx::f32x2(l1, l1), qsum2[g][nt], S2[mt][nt][x]);
            }
          if constexpr (TERMS == 1) {
#pragma unroll
            for (int j = 2 * g; j < 2 * g + 2; ++j) {
              uint32_t A[2][4];
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  A[mt][x] = kw[mt][x][j] & 0x0f0f0f0fu;
                  A[mt][2 + x] = (kw[mt][x][j] >> 4) & 0x0f0f0f0fu;
                }
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  uint32_t q2[2];
                  load_words<2>(frag[nt] + (2 * j + m) * kFragStride, q2);
#pragma unroll
                  for (int mt = 0; mt < 2; ++mt) {
                    float d[4];
                    ptx::mma_16832(d, A[mt], q2[0], q2[1]);
                    S2[mt][nt][0] = ptx::fma_f32x2(ptx::f32x2(d[0], d[1]), ks[mt][0], S2[mt][nt][0]);
                    S2[mt][nt][1] = ptx::fma_f32x2(ptx::f32x2(d[2], d[3]), ks[mt][1], S2[mt][nt][1]);
                  }
                }
            }
          } else {
            float acc[2][NT][4] = {};
#pragma unroll
            for (int jp = 4 * g; jp < 4 * g + 4; ++jp) {
              const int j = jp >> 1;
              uint32_t A[2][4];
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  A[mt][x] = jp & 1 ? nibbles<2>(kw[mt][x][j], masks) : nibble0(kw[mt][x][j], masks);
                  A[mt][2 + x] = jp & 1 ? nibbles<3>(kw[mt][x][j], masks) : nibbles<1>(kw[mt][x][j], masks);
                }
#pragma unroll
              for (int m = 0; m < TERMS; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  uint32_t q2[2];
                  load_words<2>(frag[nt] + (jp * TERMS + m) * kFragStride, q2);
#pragma unroll
                  for (int mt = 0; mt < 2; ++mt) ptx::mma_16816(acc[mt][nt], A[mt], q2[0], q2[1]);
                }
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  S2[mt][nt][x] = ptx::fma_f32x2(ptx::f32x2(acc[mt][nt][2 * x], acc[mt][nt][2 * x + 1]), ks[mt][x],
                                                 S2[mt][nt][x]);
          }
        }
      }
      // ---- P = 2^(S - ref)
      const bool masked = gone || j0 + kKv4Sub > lim_min;  // the same for the whole warp
      uint32_t vis = 0xffffffffu;  // bit (mt * NT + nt) * 4 + e: the element is visible
      if (masked) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float v[2];
              ptx::f32x2_split(S2[mt][nt][x], v[0], v[1]);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (gone || j0 + mt * 16 + x * 8 + r >= lim[nt][e]) {
                  v[e] = -INFINITY;
                  vis &= ~(1u << ((mt * NT + nt) * 4 + 2 * x + e));
                }
              S2[mt][nt][x] = ptx::f32x2(v[0], v[1]);
            }
      }
      if (a.accumulate) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              float v[2];
              ptx::f32x2_split(ptx::mul_f32x2(S2[mt][nt][x], ptx::f32x2(sl2[nt][0], sl2[nt][1])), v[0], v[1]);
              const int n = nt * 8 + 2 * c;
              float* to = gr.score + (int64_t(u) * gr.rows_per_tile + n) * kKv4Sub + mt * 16 + x * 8 + r;
              if (n < rows) to[0] = v[0];
              if (n + 1 < rows) to[kKv4Sub] = v[1];
            }
      }
      float P[2][NT][4];
      float top = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float* v = P[mt][nt] + 2 * x;
            ptx::f32x2_split(ptx::fma_f32x2(S2[mt][nt][x], ptx::f32x2(sl2[nt][0], sl2[nt][1]),
                                            ptx::f32x2(-ref[nt][0], -ref[nt][1])), v[0], v[1]);
            top = fmaxf(top, fmaxf(v[0], v[1]));
          }
      if (__any_sync(0xffffffffu, top > kSlack)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float keep[2], most[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float v[2];
              ptx::f32x2_split(ptx::mul_f32x2(S2[mt][nt][x], ptx::f32x2(sl2[nt][0], sl2[nt][1])), v[0], v[1]);
              most[0] = fmaxf(most[0], v[0]);
              most[1] = fmaxf(most[1], v[1]);
            }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = most[e];
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            m = fmaxf(m, ref[nt][e]);
            keep[e] = ptx::ex2(ref[nt][e] - m);
            ref[nt][e] = m;
          }
          const uint64_t keep2 = ptx::f32x2(keep[0], keep[1]);
          sum2[nt] = ptx::mul_f32x2(sum2[nt], keep2);
#pragma unroll
          for (int g = 0; g < GV; ++g) {
            ooff2[g][nt] = ptx::mul_f32x2(ooff2[g][nt], keep2);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int i = 0; i < 4; ++i) O[g][i][nt][e] *= keep[e & 1];
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              ptx::f32x2_split(ptx::fma_f32x2(S2[mt][nt][x], ptx::f32x2(sl2[nt][0], sl2[nt][1]),
                                              ptx::f32x2(-ref[nt][0], -ref[nt][1])), P[mt][nt][2 * x], P[mt][nt][2 * x + 1]);
        }
      }
      uint64_t P2[2][NT][2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            P2[mt][nt][x] = ptx::f32x2(ptx::ex2(P[mt][nt][2 * x]), ptx::ex2(P[mt][nt][2 * x + 1]));
            sum2[nt] = ptx::add_f32x2(sum2[nt], P2[mt][nt][x]);
          }
      // ---- O^T += V^T P^T, 16 tokens at a time
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t vw[4][GV], vs[2][(GV + 1) / 2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t tok = mt * 16 + 2 * c + (i & 1) + (i >> 1) * 8;
          load_words<GV>(st + f.vc() + tok * (DV / 2) + r * (GV * 4), vw[i]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t tok = mt * 16 + x * 8 + r;
          if constexpr (GV == 2) {
            load_words<1>(st + f.vs() + tok * 4, vs[x]);
          } else {
            vs[x][0] = __float_as_uint(load_bf16(st + f.vs() + tok * 2)) >> 16;
          }
        }
#pragma unroll
        for (int g = 0; g < GV; ++g) {
          // P s of this group as B fragments, and P low on the side
          uint32_t B0[NT][TERMS], B1[NT][TERMS];
          const float s0 = half_at(vs[0], g), s1 = half_at(vs[1], g);
          // the middle of the group's range, 8 steps up
          const float l0 = fmaf(8.f, s0, load_bf16(st + f.vl() + (g * kKv4Sub + mt * 16 + r) * 2));
          const float l1 = fmaf(8.f, s1, load_bf16(st + f.vl() + (g * kKv4Sub + mt * 16 + 8 + r) * 2));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float ps[4];
            ptx::f32x2_split(ptx::mul_f32x2(P2[mt][nt][0], ptx::f32x2(s0, s0)), ps[0], ps[1]);
            ptx::f32x2_split(ptx::mul_f32x2(P2[mt][nt][1], ptx::f32x2(s1, s1)), ps[2], ps[3]);
            if (masked) {  // what an unseen slot holds (NaN, in the worst case) reaches nothing
              float pl[4];
              ptx::f32x2_split(ptx::mul_f32x2(P2[mt][nt][0], ptx::f32x2(l0, l0)), pl[0], pl[1]);
              ptx::f32x2_split(ptx::mul_f32x2(P2[mt][nt][1], ptx::f32x2(l1, l1)), pl[2], pl[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!((vis >> ((mt * NT + nt) * 4 + e)) & 1)) ps[e] = pl[e] = 0.f;
              ooff2[g][nt] = ptx::add_f32x2(ooff2[g][nt], ptx::f32x2(pl[0] + pl[2], pl[1] + pl[3]));
            } else {
              ooff2[g][nt] = ptx::fma_f32x2(P2[mt][nt][0], ptx::f32x2(l0, l0), ooff2[g][nt]);
              ooff2[g][nt] = ptx::fma_f32x2(P2[mt][nt][1], ptx::f32x2(l1, l1), ooff2[g][nt]);
            }
            split_pair<TERMS>(ps[0], ps[1], B0[nt]);
            split_pair<TERMS>(ps[2], ps[3], B1[nt]);
#pragma unroll
            for (int m = 0; m < TERMS; ++m) {
              B0[nt][m] = ptx::movm_trans(B0[nt][m]);
              B1[nt][m] = ptx::movm_trans(B1[nt][m]);
            }
          }
          const uint32_t lo0 = __byte_perm(vw[0][g], vw[1][g], 0x5410), hi0 = __byte_perm(vw[0][g], vw[1][g], 0x7632);
          const uint32_t lo1 = __byte_perm(vw[2][g], vw[3][g], 0x5410), hi1 = __byte_perm(vw[2][g], vw[3][g], 0x7632);
          const uint32_t A[4][4] = {
              {nibble0(lo0, masks), nibble0(hi0, masks), nibble0(lo1, masks), nibble0(hi1, masks)},
              {nibbles<1>(lo0, masks), nibbles<1>(hi0, masks), nibbles<1>(lo1, masks), nibbles<1>(hi1, masks)},
              {nibbles<2>(lo0, masks), nibbles<2>(hi0, masks), nibbles<2>(lo1, masks), nibbles<2>(hi1, masks)},
              {nibbles<3>(lo0, masks), nibbles<3>(hi0, masks), nibbles<3>(lo1, masks), nibbles<3>(hi1, masks)}};
          // The tensor cores cut a sum off where they add to an accumulator. In fp32 caches each product of 16 tokens is
          // therefore added outside, rounded (96519 tokens, d 128: error of O 1.9e-7 of its norm, 9.3e-5 otherwise); in
          // bf16 caches the rounding of P s hides it (0.0024 either way at 128K tokens; 350 us, 354 outside).
          if constexpr (TERMS == 3) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float d[4] = {};
#pragma unroll
                for (int m = 0; m < TERMS; ++m) ptx::mma_16816(d, A[i], B0[nt][m], B1[nt][m]);
#pragma unroll
                for (int e = 0; e < 4; e += 2)
                  ptx::f32x2_split(ptx::add_f32x2(ptx::f32x2(O[g][i][nt][e], O[g][i][nt][e + 1]), ptx::f32x2(d[e], d[e + 1])),
                                   O[g][i][nt][e], O[g][i][nt][e + 1]);
              }
          } else {
#pragma unroll
            for (int m = 0; m < TERMS; ++m)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) ptx::mma_16816(O[g][i][nt], A[i], B0[nt][m], B1[nt][m]);
          }
        }
      }
      __syncwarp();  // the stage has been read
      if (++stage == STAGES) stage = 0;
      load_next();
      cur.next(base, a.c.num_seqs, per, row_tiles);
    }

    // ---- the warp's sums
    float sum[NT][2], ooff[GV][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ptx::f32x2_split(sum2[nt], sum[nt][0], sum[nt][1]);
#pragma unroll
      for (int g = 0; g < GV; ++g) ptx::f32x2_split(ooff2[g][nt], ooff[g][nt][0], ooff[g][nt][1]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], o);
#pragma unroll
          for (int g = 0; g < GV; ++g) ooff[g][nt][e] += __shfl_xor_sync(0xffffffffu, ooff[g][nt][e], o);
        }
    }
    const bool starts = real0 >= w0, ends = run0 + per_run <= w1;
    if (starts && ends) {  // whole: done
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int n = nt * 8 + 2 * c + e;
          if (n >= rows) continue;
          int t, head;
          const int64_t row = row_index(a, b, h, n0 + n, &t, &head);
          const float l = sum[nt][e], inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
          for (int g = 0; g < GV; ++g) {
            const float add = ooff[g][nt][e];
#pragma unroll
            for (int x = 0; x < 2; ++x)
              store_o4(a, row * DV + 64 * g + 8 * r + 4 * x,
                       make_float4((O[g][0][nt][e + 2 * x] + add) * inv, (O[g][1][nt][e + 2 * x] + add) * inv,
                                   (O[g][2][nt][e + 2 * x] + add) * inv, (O[g][3][nt][e + 2 * x] + add) * inv));
          }
          if (r == 0)
            a.lse[int64_t(head) * a.c.num_seqs * a.n_q + int64_t(b) * a.n_q + t] =
                l == 0.f ? -INFINITY : (ref[nt][e] + log2f(l)) * kLn2;
        }
    } else {
      last = !ends;
      if (last) __syncthreads();  // no ring is used any more (the other warps: below)
      float* part = (last ? last_s : stash_s) + warp * gr.rows_per_tile * DV;
      float* stat = stat_s + (2 * warp + last) * 2 * C::COLS;
      if (lane == 0) s_run[2 * warp + last] = b * per + run;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int n = nt * 8 + 2 * c + e;
          if (n >= rows) continue;
          if (r == 0) {
            stat[n] = ref[nt][e];
            stat[C::COLS + n] = sum[nt][e];
          }
#pragma unroll
          for (int g = 0; g < GV; ++g) {
            const float add = ooff[g][nt][e];
#pragma unroll
            for (int x = 0; x < 2; ++x)
              *reinterpret_cast<float4*>(part + n * DV + 64 * g + 8 * r + 4 * x) =
                  make_float4(O[g][0][nt][e + 2 * x] + add, O[g][1][nt][e + 2 * x] + add, O[g][2][nt][e + 2 * x] + add,
                              O[g][3][nt][e + 2 * x] + add);
          }
        }
    }
  }
  if (!last) __syncthreads();
  __syncthreads();

  // ---- runs cut over warps: their partials, in order, joined by the whole CTA.  First what every partial weighs:
  // lane = partial, a warp a row; partials of one run find their largest reference among them.
  constexpr int kSlots = 2 * NW;
  const int id = lane < kSlots ? s_run[lane] : -1;
  const uint32_t held = __ballot_sync(0xffffffffu, id >= 0), under = (1u << lane) - 1u;
  for (int n = warp; n < gr.rows_per_tile; n += NW) {
    float* st = stat_s + (lane < kSlots ? lane : 0) * 2 * C::COLS + n;
    const float m = id < 0 ? kNoRef : st[0], l = id < 0 ? 0.f : st[C::COLS];
    const uint32_t mask = __match_any_sync(0xffffffffu, id);
    // floats as integers of the same order
    const int order = __float_as_int(m) ^ ((__float_as_int(m) >> 31) & 0x7fffffff);
    const int top = __reduce_max_sync(mask, order);
    const float mm = __int_as_float(top ^ ((top >> 31) & 0x7fffffff));
    const float k = l == 0.f ? 0.f : ptx::ex2(m - mm);  // 0: saw nothing
    if (id >= 0) {
      st[0] = k;
      st[C::COLS] = l == 0.f ? 0.f : k * l;
      top_s[lane * C::COLS + n] = mm;
    }
  }
  if (warp == NW - 1) {
    const int before = held & under ? 31 - __clz(held & under) : -1;
    const int id_before = __shfl_sync(0xffffffffu, id, max(before, 0));
    const bool first = id >= 0 && (before < 0 || id_before != id);
    const uint32_t firsts = __ballot_sync(0xffffffffu, first);
    if (id >= 0) s_slot[__popc(held & under)] = lane;
    if (first) s_group[__popc(firsts & under)] = __popc(held & under);
    if (lane == 0) {
      s_groups = __popc(firsts);
      s_group[__popc(firsts)] = __popc(held);
    }
  }
  __syncthreads();
  // four channels of a row of a run a thread
  const int items = gr.rows_per_tile * (DV / 4);
  for (int e = tid; e < s_groups * items; e += C::THREADS) {
    const int g = e / items, n = (e - g * items) / (DV / 4), d = (e - g * items) % (DV / 4) * 4;
    const int i0 = s_group[g], i1 = s_group[g + 1], rid = s_run[s_slot[i0]];
    const int b = rid / per, run = rid - b * per;
    const int per_run = (base[b + 1] - base[b]) / per, run0 = base[b] + run * per_run;
    const int h = run / row_tiles, n0 = (run - h * row_tiles) * gr.rows_per_tile;
    if (n0 + n >= a.rows) continue;
    float l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
      const int s = s_slot[i];
      const float* st = stat_s + s * 2 * C::COLS + n;
      const float4 y = *reinterpret_cast<const float4*>(((s & 1) ? last_s : stash_s) +
                                                        ((s >> 1) * gr.rows_per_tile + n) * DV + d);
      const float k = st[0];
      l += st[C::COLS];
      x = make_float4(fmaf(k, y.x, x.x), fmaf(k, y.y, x.y), fmaf(k, y.z, x.z), fmaf(k, y.w, x.w));
    }
    const float m = top_s[s_slot[i0] * C::COLS + n];
    if (run0 + 1 >= u0 && run0 + per_run <= u1) {  // whole
      int t, head;
      const int64_t row = row_index(a, b, h, n0 + n, &t, &head);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      store_o4(a, row * DV + d, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
      if (d == 0)
        a.lse[int64_t(head) * a.c.num_seqs * a.n_q + int64_t(b) * a.n_q + t] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    } else {
      float* part = gr.part + (int64_t(blockIdx.x) * 2 + (run0 + 1 >= u0)) * part_floats(C::COLS, DV);
      *reinterpret_cast<float4*>(part + 2 * C::COLS + n * DV + d) = x;
      if (d == 0) {
        part[n] = m;
        part[C::COLS + n] = l;
      }
    }
  }
}

// Joins the runs that were cut (a CTA a row; whole ones are done, empty ones
// get o = 0, lse = -inf).
constexpr int kJoinThreads = 256;

template <int COLS, int DV>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const Kv4AttnArgs a, const Grid gr) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int32_t s_scan[kJoinThreads / 32];
  int32_t* base = reinterpret_cast<int32_t*>(smem);
  const int row_tiles = a.row_tiles, per = a.c.hkv * row_tiles;
  scan_lengths<kJoinThreads>(a, per, base, s_scan);
  const int units = base[a.c.num_seqs], shares = share_count(units, gr.ctas, gr.warps);
  ptx::grid_launch_dependents();
  ptx::grid_wait_previous();
  constexpr int kPart = part_floats(COLS, DV);
  // partial i of a run cut over shares c0, c0 + 1, ...: slot 1 of the share it starts in, slot 0 of the others
  auto part_of = [&](int c0, int i) { return gr.part + (int64_t(c0 + i) * 2 + (i == 0)) * kPart; };
  const int id = int(blockIdx.x) / gr.rows_per_tile, n = int(blockIdx.x) - id * gr.rows_per_tile;
  const int b = id / per, run = id - b * per;
  const int per_run = (base[b + 1] - base[b]) / per, run0 = base[b] + run * per_run;
  const int h = run / row_tiles, n0 = (run - h * row_tiles) * gr.rows_per_tile;
  if (n0 + n >= a.rows) return;
  int c0 = 0, parts = 0;
  if (per_run > 0) {
    c0 = share_of(units, shares, run0 + 1);
    parts = share_of(units, shares, run0 + per_run - 1) - c0 + 1;
    if (parts == 1) return;
  }
  float* k_s = reinterpret_cast<float*>(smem + gr.off_join);  // [parts]: references, then weights
  float* l_s = k_s + gr.ctas;                                 // [parts]: sums
  for (int i = threadIdx.x; i < parts; i += kJoinThreads) {
    const float* p = part_of(c0, i) + n;
    k_s[i] = p[0];
    l_s[i] = p[COLS];
  }
  __syncthreads();
  float m = kNoRef;
  for (int i = threadIdx.x & 31; i < parts; i += 32) m = fmaxf(m, k_s[i]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  __syncthreads();
  for (int i = threadIdx.x; i < parts; i += kJoinThreads) {
    const float k = l_s[i] == 0.f ? 0.f : ptx::ex2(k_s[i] - m);  // 0: saw nothing
    k_s[i] = k;
    l_s[i] = l_s[i] == 0.f ? 0.f : k * l_s[i];
  }
  __syncthreads();
  constexpr int kSplit = kJoinThreads / DV;
  float* x_s = l_s + gr.ctas;  // [kSplit][DV]
  const int d = threadIdx.x % DV, first = threadIdx.x / DV;
  float l = 0.f, x = 0.f;
#pragma unroll 8
  for (int i = first; i < parts; i += kSplit) x += k_s[i] * part_of(c0, i)[2 * COLS + n * DV + d];
  x_s[first * DV + d] = x;
  for (int i = 0; i < parts; ++i) l += l_s[i];
  __syncthreads();
  if (first > 0) return;
#pragma unroll
  for (int i = 1; i < kSplit; ++i) x += x_s[i * DV + d];
  int t, head;
  const int64_t row = row_index(a, b, h, n0 + n, &t, &head);
  store_o(a, row * DV + d, l == 0.f ? 0.f : x / l);
  if (d == 0)
    a.lse[int64_t(head) * a.c.num_seqs * a.n_q + int64_t(b) * a.n_q + t] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Adds up the weights: a warp takes consecutive sub-blocks, of a kv head at a
// time, a lane a token.  The scores come from L2, the lse from the kernels
// before; every slot gets one sum a row tile, in order.
__global__ void __launch_bounds__(kJoinThreads, 5) kv4_weights_kernel(const Kv4AttnArgs a, const Grid gr) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int32_t s_scan[kJoinThreads / 32];
  int32_t* base = reinterpret_cast<int32_t*>(smem);
  const int row_tiles = a.row_tiles, per = a.c.hkv * row_tiles;
  scan_lengths<kJoinThreads>(a, per, base, s_scan);
  const int units = base[a.c.num_seqs];
  ptx::grid_wait_previous();
  const int lane = threadIdx.x & 31;
  const int warps = int(gridDim.x) * (kJoinThreads / 32);
  const int w = int(blockIdx.x) * (kJoinThreads / 32) + int(threadIdx.x >> 5);
  const int all = units / row_tiles;  // units of the cache: row tile by row tile the same
  const int each = (all + warps - 1) / warps;
  const int v1 = int(min(int64_t(all), int64_t(each) * (w + 1)));
  int b = 0;
  for (int v = int(min(int64_t(all), int64_t(each) * w)); v < v1;) {
    b = seq_of_unit(base, a.c.num_seqs, b, v * row_tiles);
    const int per_run = (base[b + 1] - base[b]) / per;
    const int at = v - base[b] / row_tiles, h = at / per_run, first = at - h * per_run;
    const int i0 = max(first - 1, 0), i1 = min(per_run, first + v1 - v) - 1;  // sub-blocks
    v += per_run - first;
    const int len = kv4_length(a.c, a.lengths, b);
    for (int rt = 0; rt < row_tiles; ++rt) {
      const int run0 = base[b] + (h * row_tiles + rt) * per_run, n0 = rt * gr.rows_per_tile;
      const int rows = min(gr.rows_per_tile, a.rows - n0);
      float ls = INFINITY;  // lane n: the lse of row n (log2)
      if (lane < rows) {
        int t, head;
        row_index(a, b, h, n0 + lane, &t, &head);
        ls = a.lse[int64_t(head) * a.c.num_seqs * a.n_q + int64_t(b) * a.n_q + t] * kLog2e;
      }
      if (ls == -INFINITY) ls = INFINITY;  // a row that sees nothing gives nothing
      const bool any_nan = __any_sync(0xffffffffu, ls != ls);
      for (int i = i0; i < i1; i += 4) {
        float add[4] = {0.f, 0.f, 0.f, 0.f};
        int page[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          page[k] = __ldg(a.c.table + int64_t(b) * a.c.max_pages + min(i + k, i1 - 1) / (CP_KV4_PAGE / kKv4Sub));
        const float* sc = gr.score + int64_t(run0 + 1 + i) * gr.rows_per_tile * kKv4Sub + lane;
        auto add_rows = [&](auto nan_) {
#pragma unroll 4
          for (int n = 0; n < rows; ++n) {
            const float lsn = __shfl_sync(0xffffffffu, ls, n);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (i + k < i1) {
                const float x = sc[(k * gr.rows_per_tile + n) * kKv4Sub];
                if (!decltype(nan_)::value || x != -INFINITY) add[k] += ptx::ex2(x - lsn);
              }
          }
        };
        // a row whose lse is NaN gives the slots that it does not see nothing all the same
        if (any_nan) add_rows(std::true_type{});
        else add_rows(std::false_type{});
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int slot = (i + k) * kKv4Sub + lane;
          if (i + k >= i1 || slot >= len) continue;
          const int pg = page[k];
          if (pg < 0 || pg >= a.c.num_pages) continue;  // (recorded by the first kernel)
          atomicAdd(a.c.weights + (int64_t(pg) * a.c.hkv + h) * CP_KV4_PAGE + slot % CP_KV4_PAGE, add[k]);
        }
      }
    }
  }
}

// Rows of one pass: up to 8 in one column tile of the MMAs, else up to 16 in
// two (fp32 caches: 8, their three terms take the registers).
int cols_of(int rows, int dtype) { return dtype == CP_DT_BF16 && rows > 8 ? 16 : 8; }

uint32_t up(uint32_t x, uint32_t n) { return (x + n - 1) / n * n; }

constexpr uint32_t kMostShared = 230000;  // 227 KB less the static arrays

// Shared memory of the first kernel: fills in the offsets, returns the bytes.
template <typename C>
uint32_t shared_layout(int num_seqs, Grid& gr) {
  uint32_t off = 0;
  gr.off_base = off;
  off = up(off + 4 * (num_seqs + 1), 128);
  gr.off_frag = off;
  off += C::NW * (C::DQK / 16 * C::TERMS * 32) * C::COLS;
  gr.off_stat = off;
  off += 2 * C::NW * 3 * C::COLS * 4;
  gr.off_stash = off;
  const uint32_t partials = C::NW * gr.rows_per_tile * C::DV * 4;
  off = up(off + partials, 128);
  gr.off_ring = off;
  // the rings hold the last partials in the end
  return off + std::max<uint32_t>(C::STAGES * C::NW * C::SUB, partials);
}

// Calls f with the configuration for these head dims, columns and type.
template <int DQK, int DV, typename F>
auto with_config(int cols, int dtype, F f) {
  if (dtype == CP_DT_F32) return f(Cfg<DQK, DV, 1, 3, 8>{});
  if (cols == 16) return f(Cfg<DQK, DV, 2, 1, 8>{});
  // twelve warps: three a scheduler (sixteen would leave 128 registers a thread, and spill; measured with ten, twelve,
  // fourteen and sixteen: 400, 345, 401 us and no room at 128K tokens of 64 heads 192 / 128)
  return f(Cfg<DQK, DV, 1, 1, 12>{});
}
template <typename F>
auto with_dims(int dqk, int dv, int cols, int dtype, F f) {
  switch (dqk * 1000 + dv) {
    case 64064: return with_config<64, 64>(cols, dtype, f);
    case 64128: return with_config<64, 128>(cols, dtype, f);
    case 128064: return with_config<128, 64>(cols, dtype, f);
    case 192064: return with_config<192, 64>(cols, dtype, f);
    case 192128: return with_config<192, 128>(cols, dtype, f);
    default: return with_config<128, 128>(cols, dtype, f);
  }
}

template <typename C, typename E>
cudaError_t launch(const Kv4AttnArgs& a, Grid gr, cudaStream_t st) {
  const uint32_t bytes = shared_layout<C>(a.c.num_seqs, gr);
  if (bytes > kMostShared) return cudaErrorInvalidValue;
  gr.warps = C::NW;
  auto kernel = kv4_attn_kernel<C, E>;
  static std::atomic<uint64_t> ready{0};  // devices whose kernel may use that much shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostShared));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  kernel<<<unsigned(gr.ctas), C::THREADS, bytes, st>>>(a, gr);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int runs = a.c.num_seqs * a.c.hkv * a.row_tiles;
  gr.off_join = up(4 * (a.c.num_seqs + 1), 16);
  const uint32_t join_smem = gr.off_join + (2 * gr.ctas + kJoinThreads) * 4;
  // the launches overlap the kernel before: they wait on the device
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(runs * gr.rows_per_tile));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = join_smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_join_kernel<C::COLS, C::DV>, a, gr);
  if (e != cudaSuccess) return e;
  if (a.accumulate) {
    cfg.gridDim = dim3(unsigned(5 * gr.ctas));
    cfg.dynamicSmemBytes = gr.off_join;
    e = cudaLaunchKernelEx(&cfg, kv4_weights_kernel, a, gr);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

struct Layout {
  int rows, cols, row_tiles, rows_per_tile;
  size_t part, score, total;
};
Layout layout_of(int num_seqs, int hq, int hkv, int dqk, int dv, int max_pages, int dtype, int n_q, int accumulate) {
  Layout L;
  L.rows = hq / hkv * n_q;
  L.cols = cols_of(L.rows, dtype);
  L.row_tiles = (L.rows + L.cols - 1) / L.cols;
  for (;; ++L.row_tiles) {  // more passes of fewer rows where their partials do not fit (many sequences, wide heads)
    L.rows_per_tile = (L.rows + L.row_tiles - 1) / L.row_tiles;
    Grid gr{};
    gr.rows_per_tile = L.rows_per_tile;
    const uint32_t bytes = with_dims(dqk, dv, L.cols, dtype, [&](auto c) { return shared_layout<decltype(c)>(num_seqs, gr); });
    if (bytes <= kMostShared || L.rows_per_tile == 1) break;
  }
  L.row_tiles = (L.rows + L.rows_per_tile - 1) / L.rows_per_tile;
  L.part = 0;
  L.score = (size_t(kv4_sm_count()) * 2 * part_floats(L.cols, dv) * 4 + 255) / 256 * 256;
  const size_t units = size_t(num_seqs) * hkv * L.row_tiles * (size_t(max_pages) * (CP_KV4_PAGE / kKv4Sub) + 1);
  L.total = L.score + (accumulate ? units * L.rows_per_tile * kKv4Sub * 4 : 0);
  L.total = (L.total + 255) / 256 * 256;
  return L;
}
Layout layout_of(const cp_kv4_t* c, int n_q, int accumulate) {
  return layout_of(c->num_seqs, c->hq, c->hkv, c->d_qk, c->d_v, c->max_pages, c->dtype, n_q, accumulate);
}

}  // namespace

int kv4_sm_count() {
  static std::atomic<int> counts[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  n = counts[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
    counts[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

size_t kv4_attn_workspace(const cp_kv4_t* c, int32_t n_q, int32_t accumulate) {
  return layout_of(c, n_q, accumulate).total;
}

int64_t kv4_attn_units(const cp_kv4_t* c, int32_t n_q) {
  return int64_t(c->num_seqs) * c->hkv * (int64_t(c->max_pages) * (CP_KV4_PAGE / kKv4Sub) + 1) * layout_of(c, n_q, 0).row_tiles;
}

cudaError_t launch_kv4_attn(Kv4AttnArgs a, int dqk, int dv, int dtype, cudaStream_t st) {
  const Layout L = layout_of(a.c.num_seqs, a.c.hq, a.c.hkv, dqk, dv, a.c.max_pages, dtype, a.n_q, a.accumulate);
  a.rows = L.rows;
  a.row_tiles = L.row_tiles;
  Grid gr{};
  gr.ctas = kv4_sm_count();
  gr.rows_per_tile = L.rows_per_tile;
  gr.part = reinterpret_cast<float*>(a.ws + L.part);
  gr.score = reinterpret_cast<float*>(a.ws + L.score);
  return with_dims(dqk, dv, L.cols, dtype, [&](auto c) {
    using C = decltype(c);
    if constexpr (C::TERMS == 3) return launch<C, float>(a, gr, st);
    else return launch<C, __nv_bfloat16>(a, gr, st);
  });
}

}  // namespace cpattn
