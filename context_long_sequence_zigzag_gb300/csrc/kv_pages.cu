// kv_pages.cu — pages that several sequences hold: room for new tokens, forks
// (shared pages, copies of those that are written), compaction, copies.
//
// The bookkeeping is a scan over refs (4 bytes a page) in page order, so that
// free pages come out lowest first: a cluster of eight CTAs counts its eighths,
// exchanges the counts through distributed shared memory and gives every free
// page its rank.  A sequence's demand is a prefix sum over the batch, so the
// page of rank r finds its taker by binary search: no free list, no atomics on
// a counter, the same answer every time.  Copies follow in a kernel of their
// own over all SMs, from a list of pairs that the scan leaves in the workspace.
#include <algorithm>

#include <cooperative_groups.h>

#include "kv.cuh"
#include "sm103_ptx.cuh"

namespace cpattn {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPerWarp = 4;                            // pages a lane of a step
constexpr int kStep = kThreads * kPerWarp;             // pages of a step of a CTA
constexpr int kMostSeqs = CP_KV4_MAX_SEQS;
// Entries of a fork's tables that the cluster that takes the pages does itself: one a thread.  It saves a launch (2 to 3 us
// of the host) and takes as long on the device (4K entries 6.8 us, with a kernel of their own 6.5); 32K entries 9.5 us against
// 6.4, 260K 36 us against 10.
constexpr int kFewEntries = kCluster * kThreads;

// Head of the workspace; the lists follow (src, then dst).
struct PairList {
  int32_t n;
  int32_t pad[63];
};
static_assert(sizeof(PairList) == 256, "PairList layout");

int64_t list_rows(int32_t num_pages, int32_t num_seqs) { return std::max<int64_t>(num_pages / 2 + 1, num_seqs); }

__device__ __forceinline__ int32_t pages_of(int64_t tokens, int32_t page_size) {
  return int32_t((tokens + page_size - 1) / page_size);
}

// Exclusive prefix sum of one value a thread over the CTA; *total: the sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(~0u, y, d);
    if (lane >= d) y += z;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = y;
  __syncthreads();
  const int w = warp_sums[lane];
  int s = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(~0u, s, d);
    if (lane >= d) s += z;
  }
  *total = __shfl_sync(~0u, s, 31);
  return y - x + __shfl_sync(~0u, s - w, warp);
}

// n numbers to their exclusive prefix sums, x[n] the sum, which is returned.
__device__ __forceinline__ int to_prefix(int32_t* x, int n, int* warp_sums) {
  int sum = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + threadIdx.x;
    int total;
    const int before = block_scan(i < n ? x[i] : 0, warp_sums, &total);
    if (i < n) x[i] = sum + before;
    sum += total;
  }
  if (threadIdx.x == 0) x[n] = sum;
  __syncthreads();
  return sum;
}

// The last of x[0 .. n - 1] (n > 0, ascending from 0) that is at most y.
__device__ __forceinline__ int last_at_most(const int32_t* x, int n, int y) {
  int a = 0, b = n - 1;
  while (a < b) {
    const int mid = (a + b + 1) >> 1;
    if (x[mid] <= y) a = mid;
    else b = mid - 1;
  }
  return a;
}

// Refs of the CTA's part of the pool, in order: f(page, refs, rank) for every
// page of [lo, hi) with pick(page, refs); rank counts them from `rank0` on.
// Stops once `most` ranks are given.  Returns the number picked (in all threads).
template <typename Pick, typename F>
__device__ __forceinline__ int scan_refs(const int32_t* refs, int lo, int hi, int rank0, int most, int* warp_sums,
                                         Pick pick, F f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int got = 0;
  for (int base = lo; base < hi && rank0 + got < most; base += kStep) {
    const int p0 = base + warp * (32 * kPerWarp) + lane;
    int32_t r[kPerWarp];
    unsigned in[kPerWarp];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kPerWarp; ++k) r[k] = p0 + 32 * k < hi ? __ldcg(refs + p0 + 32 * k) : 0;
#pragma unroll
    for (int k = 0; k < kPerWarp; ++k) {
      in[k] = __ballot_sync(~0u, p0 + 32 * k < hi && pick(p0 + 32 * k, r[k]));
      mine += __popc(in[k]);
    }
    __syncthreads();
    if (lane == 0) warp_sums[warp] = mine;
    __syncthreads();
    int s = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int z = __shfl_up_sync(~0u, s, d);
      if (lane >= d) s += z;
    }
    const int below = __shfl_sync(~0u, s, (warp + 31) & 31);
    int rank = rank0 + got + (warp ? below : 0);
#pragma unroll
    for (int k = 0; k < kPerWarp; ++k) {
      if (in[k] >> lane & 1) f(p0 + 32 * k, r[k], rank + __popc(in[k] & ((1u << lane) - 1)));
      rank += __popc(in[k]);
    }
    got += __shfl_sync(~0u, s, 31);
  }
  return got;
}

// The CTA's part of n pages.
__device__ __forceinline__ void part_of(int n, int cta, int* lo, int* hi) {
  const int steps = (n + kStep - 1) / kStep;
  *lo = min(n, int(int64_t(steps) * cta / kCluster) * kStep);
  *hi = min(n, int(int64_t(steps) * (cta + 1) / kCluster) * kStep);
}

// Every CTA's two counts, summed below this CTA's and over all.
struct Sums {
  int below[2], all[2];
};
__device__ __forceinline__ Sums exchange(cg::cluster_group& cluster, int (*counts)[2], int cta, int x, int y) {
  if (threadIdx.x < kCluster) {
    int* there = cluster.map_shared_rank(&counts[cta][0], threadIdx.x);
    there[0] = x, there[1] = y;
  }
  cluster.sync();
  Sums s{};
  for (int i = 0; i < kCluster; ++i)
    for (int k = 0; k < 2; ++k) {
      s.all[k] += counts[i][k];
      if (i < cta) s.below[k] += counts[i][k];
    }
  return s;
}

// What a batch asks for: pages for entries first[b] .. of row b.
struct Demand {
  int32_t* table;
  int32_t num_seqs, max_pages, page_size;
  const int32_t* lengths;
  const int32_t* extra;  // reserve: tokens to come, or to go
};

// What a fork starts from and leaves.
struct Fork {
  PageTable old;
  const int32_t* parents;
  int32_t* new_lengths;
};

// The old sequences let go of their pages, the new ones (of `d`) take theirs; a page held in part is counted later.
// Thread i of n.
__device__ __forceinline__ void fork_rows(int32_t* refs, int32_t num_pages, const Fork& f, const Demand& d, int64_t i0,
                                          int64_t n, int32_t* err) {
  const int64_t most = int64_t(f.old.max_pages) * d.page_size, new_most = int64_t(d.max_pages) * d.page_size;
  for (int64_t i = i0; i < int64_t(f.old.num_seqs) * f.old.max_pages; i += n) {
    const int b = int(i / f.old.max_pages), e = int(i - int64_t(b) * f.old.max_pages);
    if (e >= pages_of(kv_length(__ldg(f.old.lengths + b), most, err), d.page_size)) continue;
    const int32_t p = kv_page(__ldg(f.old.table + i), num_pages, err);
    if (p >= 0) atomicSub(refs + p, 1);
  }
  const int across = max(d.max_pages, 1);  // (a length is written even where no page is)
  for (int64_t i = i0; i < int64_t(d.num_seqs) * across; i += n) {
    const int b = int(i / across), e = int(i - int64_t(b) * across);
    int32_t from = __ldg(f.parents + b);
    if (from >= f.old.num_seqs) {
      kv_error(err, kKvSlot);
      from = -1;
    }
    int32_t len = from >= 0 ? kv_length(__ldg(f.old.lengths + from), most, nullptr) : 0;
    if (len > new_most) {
      kv_error(err, kKvLength);
      len = int32_t(new_most);
    }
    if (e == 0) f.new_lengths[b] = len;
    if (e >= d.max_pages) continue;
    int32_t p = -1;
    if (e < pages_of(len, d.page_size)) {
      p = __ldg(f.old.table + int64_t(from) * f.old.max_pages + e);
      if (p < 0 || p >= num_pages) p = -1;  // (recorded above)
      else if (e < len / d.page_size) atomicAdd(refs + p, 1);
    }
    d.table[int64_t(b) * d.max_pages + e] = p;
  }
}

__global__ void __launch_bounds__(256)
    pages_rows_kernel(int32_t* refs, int32_t num_pages, Fork f, Demand d, int32_t* err) {
  ptx::grid_launch_dependents();
  fork_rows(refs, num_pages, f, d, int64_t(blockIdx.x) * 256 + threadIdx.x, int64_t(gridDim.x) * 256, err);
}

// Shared memory: first [num_seqs] (padded to four), prefix [num_seqs + 1].  FORK, `rows`: the rows are done here, not by
// a kernel before.
template <bool FORK>
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
    pages_take_kernel(int32_t* refs, int32_t num_pages, Fork f, int32_t rows, Demand d, int32_t* counts, PairList* list,
                      int32_t* src, int32_t* dst, int32_t* err) {
  extern __shared__ __align__(16) int32_t shared[];
  __shared__ int warp_sums[kWarps];
  __shared__ int cta_counts[kCluster][2];
  cg::cluster_group cluster = cg::this_cluster();
  const int cta = int(cluster.block_rank()), tid = threadIdx.x;
  int32_t* first = shared;
  int32_t* prefix = shared + (d.num_seqs + 3) / 4 * 4;
  int lo, hi;
  part_of(num_pages, cta, &lo, &hi);

  if constexpr (FORK) {
    if (rows) {
      fork_rows(refs, num_pages, f, d, cta * kThreads + tid, kCluster * kThreads, err);
      cluster.sync();
    } else {
      ptx::grid_wait_previous();
    }
    // the page that sequence b holds in part, -1: none
    for (int b = tid; b < d.num_seqs; b += kThreads) {
      const int32_t n = __ldcg(d.lengths + b);
      first[b] = n % d.page_size ? __ldcg(d.table + int64_t(b) * d.max_pages + n / d.page_size) : -1;
    }
    __syncthreads();
    bool keeps[kMostSeqs / kThreads];
#pragma unroll
    for (int k = 0; k < kMostSeqs / kThreads; ++k) {
      const int b = tid + k * kThreads;
      keeps[k] = false;
      if (b >= d.num_seqs) continue;
      const int32_t p = first[b];
      bool earlier = false;
      if (p >= 0) {
        keeps[k] = __ldcg(refs + p) == 0;
        for (int i = 0; i < b / 4; ++i) {
          const int4 x = reinterpret_cast<const int4*>(first)[i];
          earlier = earlier || x.x == p || x.y == p || x.z == p || x.w == p;
        }
        for (int i = b & ~3; i < b; ++i) earlier = earlier || first[i] == p;
      }
      keeps[k] = keeps[k] && !earlier;
      prefix[b] = p >= 0 && !keeps[k];
    }
    cluster.sync();  // every CTA has read refs
    // (a page is scanned by one CTA, which marks it)
#pragma unroll
    for (int k = 0; k < kMostSeqs / kThreads; ++k) {
      const int32_t p = keeps[k] ? first[tid + k * kThreads] : -1;
      if (p >= lo && p < hi) __stcg(refs + p, 1);
    }
    __syncthreads();
  } else {
    int32_t demand[kMostSeqs / kThreads];
    bool gone = false;
#pragma unroll
    for (int k = 0; k < kMostSeqs / kThreads; ++k) {
      const int b = tid + k * kThreads;
      demand[k] = 0;
      if (b >= d.num_seqs) continue;
      const int64_t most = int64_t(d.max_pages) * d.page_size;
      const int32_t n = kv_length(__ldg(d.lengths + b), most, err);
      const int64_t want = max(int64_t(n) + __ldg(d.extra + b), int64_t(0));
      if (want > most) kv_error(err, kKvLength);
      const int32_t held = pages_of(n, d.page_size), needs = pages_of(min(want, most), d.page_size);
      first[b] = held;
      prefix[b] = max(held - needs, 0);
      demand[k] = max(needs - held, 0);
      gone = gone || needs < held;
    }
    // What shorter sequences let go of: an entry a thread of the cluster, by a prefix sum over the batch (8192 pages of
    // one sequence: 8.9 us for the call, 512 of 64 sequences 13; a thread a sequence: 656 and 87 us).
    if (__syncthreads_or(gone)) {
      const int all = to_prefix(prefix, d.num_seqs, warp_sums);
      for (int i = cta * kThreads + tid; i < all; i += kCluster * kThreads) {
        const int b = last_at_most(prefix, d.num_seqs, i);
        int32_t* entry = d.table + int64_t(b) * d.max_pages + first[b] - 1 - (i - prefix[b]);
        const int32_t p = kv_page(*entry, num_pages, err);
        if (p >= 0) atomicSub(refs + p, 1);
        *entry = -1;
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kMostSeqs / kThreads; ++k)
      if (tid + k * kThreads < d.num_seqs) prefix[tid + k * kThreads] = demand[k];
    cluster.sync();  // before the free pages are counted, and shared memory is written from other CTAs
  }
  const int wanted = to_prefix(prefix, d.num_seqs, warp_sums);

  auto is_free = [](int, int32_t r) { return r == 0; };
  const int free_here = scan_refs(refs, lo, hi, 0, INT32_MAX, warp_sums, is_free, [](int, int32_t, int) {});
  // (hi - lo less the free ones includes negative counts of a caller's mistake: in use, as they are not free)
  const Sums s = exchange(cluster, cta_counts, cta, free_here, hi - lo - free_here);
  const int given = min(wanted, s.all[0]);
  auto taker = [&](int rank) { return last_at_most(prefix, d.num_seqs, rank); };
  auto entry_of = [&](int b, int rank) {
    const int e = FORK ? __ldcg(d.lengths + b) / d.page_size : first[b] + rank - prefix[b];
    return d.table + int64_t(b) * d.max_pages + e;
  };
  if (s.below[0] < given)
    scan_refs(refs, lo, hi, s.below[0], given, warp_sums, is_free, [&](int page, int32_t, int rank) {
      if (rank >= given) return;
      const int b = taker(rank);
      if (FORK) src[rank] = first[b], dst[rank] = page;
      *entry_of(b, rank) = page;
      refs[page] = 1;
    });
  for (int rank = given + cta * kThreads + tid; rank < wanted; rank += kCluster * kThreads) {
    const int b = taker(rank);
    *entry_of(b, rank) = -1;
    kv_error(err, kKvNoPage);
  }
  if (cta == 0 && tid == 0) {
    if (FORK) list->n = given;
    counts[0] = s.all[1] + given;
    counts[1] = wanted - given;
  }
}

// Compaction: holes below the number of pages in use and the pages behind it,
// each in order, meet in the lists.
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
    pages_pack_kernel(int32_t* refs, int32_t num_pages, int32_t* moved, int32_t* counts, PairList* list, int32_t* src,
                      int32_t* dst) {
  __shared__ int warp_sums[kWarps];
  __shared__ int cta_counts[2][kCluster][2];
  cg::cluster_group cluster = cg::this_cluster();
  const int cta = int(cluster.block_rank());
  cluster.barrier_arrive();  // all are there before their shared memory is written (the wait is below)
  int lo, hi;
  part_of(num_pages, cta, &lo, &hi);
  auto nothing = [](int, int32_t, int) {};
  const int free_here = scan_refs(refs, lo, hi, 0, INT32_MAX, warp_sums, [](int, int32_t r) { return r == 0; }, nothing);
  cluster.barrier_wait();
  const int used = exchange(cluster, cta_counts[0], cta, free_here, hi - lo - free_here).all[1];
  // free pages of this part below `used` and used ones behind it; only the part that it lies in has to look
  int holes = lo < used ? free_here : 0;
  if (lo < used && used < hi)
    holes = scan_refs(refs, lo, used, 0, INT32_MAX, warp_sums, [](int, int32_t r) { return r == 0; }, nothing);
  const int movers = hi - lo - free_here - (min(max(used, lo), hi) - lo - holes);
  const Sums s = exchange(cluster, cta_counts[1], cta, holes, movers);
  // in page order the part's holes come before its movers
  scan_refs(
      refs, lo, hi, 0, INT32_MAX, warp_sums,
      [&](int p, int32_t r) {
        if (p < used || r == 0) moved[p] = r ? p : -1;
        return p < used ? r == 0 : r != 0;
      },
      [&](int p, int32_t, int rank) {
        if (p < used) __stcg(dst + s.below[0] + rank, p);
        else __stcg(src + s.below[1] + rank - holes, p);
      });
  cluster.sync();
  for (int i = cta * kThreads + threadIdx.x; i < s.all[1]; i += kCluster * kThreads) {
    const int32_t from = __ldcg(src + i), to = __ldcg(dst + i);
    moved[from] = to;
    refs[to] = __ldcg(refs + from);
    refs[from] = 0;
  }
  if (cta == 0 && threadIdx.x == 0) {
    list->n = s.all[1];
    counts[0] = used;
    counts[1] = 0;
  }
}

// A table follows the pages' moves.
struct Follow {
  PageTable t;
  int32_t page_size;
  const int32_t* moved;
  int32_t* new_table;  // nullptr: no table
};

constexpr int kCopyThreads = 256;
constexpr int kChunk = kCopyThreads * 16 * 4;

// Pages of all buffers, by pieces of 16 KiB: four loads a thread, then four stores.
__global__ void __launch_bounds__(kCopyThreads)
    pages_copy_kernel(const __grid_constant__ PageBuffers b, const int32_t* n_dev, int32_t n_host, const int32_t* src,
                      const int32_t* dst, Follow fo, int32_t* err) {
  __shared__ int32_t chunk0[CP_PAGES_MAX_BUFFERS + 1];
  if (threadIdx.x == 0) {
    int at = 0;
    for (int i = 0; i < b.n; ++i) {
      chunk0[i] = at;
      at += int((b.bytes[i] + kChunk - 1) / kChunk);
    }
    chunk0[b.n] = at;
  }
  __syncthreads();
  if (n_dev) ptx::grid_wait_previous();
  if (fo.new_table) {
    const int64_t all = int64_t(fo.t.num_seqs) * fo.t.max_pages, most = int64_t(fo.t.max_pages) * fo.page_size;
    for (int64_t i = int64_t(blockIdx.x) * kCopyThreads + threadIdx.x; i < all; i += int64_t(gridDim.x) * kCopyThreads) {
      const int s = int(i / fo.t.max_pages), e = int(i - int64_t(s) * fo.t.max_pages);
      int32_t p = -1;
      if (e < pages_of(kv_length(__ldg(fo.t.lengths + s), most, err), fo.page_size)) {
        p = kv_page(fo.t.table[i], b.num_pages[0], err);
        if (p >= 0) p = __ldcg(fo.moved + p);
      }
      fo.new_table[i] = p;
    }
  }
  const int n = n_dev ? __ldcg(n_dev) : n_host;
  const int per = chunk0[b.n];
  for (int64_t it = blockIdx.x; it < int64_t(n) * per; it += gridDim.x) {
    const int pair = int(it / per), c = int(it - int64_t(pair) * per);
    int32_t from = __ldcg(src + pair), to = __ldcg(dst + pair);
    if (n_dev == nullptr) {  // a caller's pairs
      if (from < 0 || to < 0) continue;
      from = kv_page(from, b.num_pages[0], threadIdx.x == 0 ? err : nullptr);
      to = kv_page(to, b.num_pages[1], threadIdx.x == 0 ? err : nullptr);
      if (from < 0 || to < 0) continue;
    }
    int x = 0, y = b.n - 1;  // the last buffer that starts at or before c
    while (x < y) {
      const int mid = (x + y + 1) >> 1;
      if (chunk0[mid] <= c) x = mid;
      else y = mid - 1;
    }
    const int64_t bytes = b.bytes[x], off = int64_t(c - chunk0[x]) * kChunk + threadIdx.x * 16;
    const char* in = b.from[x] + from * bytes;
    char* out = b.to[x] + to * bytes;
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (off + k * kCopyThreads * 16 < bytes) v[k] = __ldcs(reinterpret_cast<const uint4*>(in + off + k * kCopyThreads * 16));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (off + k * kCopyThreads * 16 < bytes) __stcs(reinterpret_cast<uint4*>(out + off + k * kCopyThreads * 16), v[k]);
  }
}

// Launches that may start before the kernel ahead of them is done (they wait on the device).
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t st,
                          A... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct Lists {
  PairList* head;
  int32_t* src;
  int32_t* dst;
};
Lists lists_of(char* ws, int32_t num_pages, int32_t num_seqs) {
  Lists l;
  l.head = reinterpret_cast<PairList*>(ws);
  l.src = reinterpret_cast<int32_t*>(ws + sizeof(PairList));
  l.dst = l.src + list_rows(num_pages, num_seqs);
  return l;
}

size_t take_smem(int32_t num_seqs) { return (size_t(num_seqs + 3) / 4 * 4 + num_seqs + 1) * 4; }

unsigned copy_grid() { return unsigned(8 * sm_count()); }

}  // namespace

size_t pages_workspace(int32_t num_pages, int32_t num_seqs) {
  return (sizeof(PairList) + size_t(list_rows(num_pages, num_seqs)) * 8 + 255) / 256 * 256;
}

cudaError_t launch_pages_reserve(int32_t num_pages, int32_t page_size, int32_t* refs, PageTable t, int32_t* table,
                                 const int32_t* extra, int32_t* counts, int32_t* err, cudaStream_t st) {
  const Demand d{table, t.num_seqs, t.max_pages, page_size, t.lengths, extra};
  pages_take_kernel<false><<<kCluster, kThreads, take_smem(t.num_seqs), st>>>(refs, num_pages, Fork{}, 0, d, counts,
                                                                             nullptr, nullptr, nullptr, err);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PageBuffers& b, int32_t page_size, int32_t* refs, PageTable t, int32_t new_seqs,
                              int32_t new_max_pages, const int32_t* parents, int32_t* new_table, int32_t* new_lengths,
                              int32_t* counts, char* ws, int32_t* err, cudaStream_t st) {
  const int32_t num_pages = b.num_pages[0];
  const Lists l = lists_of(ws, num_pages, std::max(t.num_seqs, new_seqs));
  const Fork f{t, parents, new_lengths};
  const Demand d{new_table, new_seqs, new_max_pages, page_size, new_lengths, nullptr};
  const int64_t entries = int64_t(t.num_seqs) * t.max_pages + int64_t(new_seqs) * std::max(new_max_pages, 1);
  const bool few = entries <= kFewEntries;
  cudaError_t e;
  if (few) {
    pages_take_kernel<true><<<kCluster, kThreads, take_smem(new_seqs), st>>>(refs, num_pages, f, 1, d, counts, l.head,
                                                                            l.src, l.dst, err);
    e = cudaGetLastError();
  } else {
    const unsigned grid = unsigned(std::clamp<int64_t>((entries + 255) / 256, 1, 8 * sm_count()));
    pages_rows_kernel<<<grid, 256, 0, st>>>(refs, num_pages, f, d, err);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_behind(pages_take_kernel<true>, kCluster, kThreads, take_smem(new_seqs), st, refs, num_pages, f, 0, d,
                      counts, l.head, l.src, l.dst, err);
  }
  if (e != cudaSuccess || b.n == 0) return e;
  return launch_behind(pages_copy_kernel, copy_grid(), kCopyThreads, 0, st, b, &l.head->n, 0, l.src, l.dst, Follow{},
                       err);
}

cudaError_t launch_pages_compact(const PageBuffers& b, int32_t page_size, int32_t* refs, PageTable t,
                                 int32_t* new_table, int32_t* moved, int32_t* counts, char* ws, int32_t* err,
                                 cudaStream_t st) {
  const Lists l = lists_of(ws, b.num_pages[0], t.num_seqs);
  pages_pack_kernel<<<kCluster, kThreads, 0, st>>>(refs, b.num_pages[0], moved, counts, l.head, l.src, l.dst);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const Follow fo{t, page_size, moved, t.num_seqs && t.max_pages ? new_table : nullptr};
  return launch_behind(pages_copy_kernel, copy_grid(), kCopyThreads, 0, st, b, &l.head->n, 0, l.src, l.dst, fo, err);
}

cudaError_t launch_pages_copy(const PageBuffers& b, int32_t n, const int32_t* src, const int32_t* dst, int32_t* err,
                              cudaStream_t st) {
  pages_copy_kernel<<<copy_grid(), kCopyThreads, 0, st>>>(b, nullptr, n, src, dst, Follow{}, err);
  return cudaGetLastError();
}

}  // namespace cpattn
