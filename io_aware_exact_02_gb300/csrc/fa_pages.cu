// fa_pages.cu -- the pages of a paged cache as a whole: copying them, forking
// sequences (whole pages shared, the last one copied), freeing them, and
// compacting the pool.
//
// A page number stands for the same page in every cache of a model, so a page is
// copied in all of them.  refs[p] counts the sequences that hold page p; 0 is a
// free page.  What is free or in use is found by a scan of refs, in ranges of
// kRange pages to a CTA:
//     used(p) = the pages in use below p,    free(p) = p - used(p).
// A fork takes the k-th lowest free page for its k-th child with a page that is
// not full.  A compaction of `live` pages in use moves the k-th highest of those
// at or past `live` (k = live - 1 - used(p)) to the k-th lowest free one: each
// source lies behind every destination, so pages are moved in any order.
//
// Two launches each (three where the scan takes several CTAs): the plan, bound by
// its latencies, and the copying with the bookkeeping, bound by memory.
// Measured: 256 children of 64 sequences, a page of 32 KB in each of 16 caches: fork
// and release 34 us (268 MB moved, a parent's page read from L2 but once); half of
// 2.2 GB moved down in 201 us (6.2 TB/s of the 6.8 that a copy reaches); small calls 6
// to 7 us.
#include <algorithm>

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_pages.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 1024;      // of the plan
constexpr int kPer = kPagesRange / kThreads;
constexpr int kCopyThreads = 256;
constexpr int kCopyEach = 4;        // 16-byte pieces of a thread in flight
constexpr int kChunk = kCopyThreads * kCopyEach * 16;

__device__ __forceinline__ void report(int* status, int site) {
  int abort_flag = 0;
  report_status(status, &abort_flag, FA_ERR_PAGE, site);
}

// Exclusive prefix sum over the CTA's kThreads threads; `all`: the sum.
__device__ __forceinline__ int block_scan(int x, int& all) {
  __shared__ int sums[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // (the last scan's sums were read)
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int before = 0;
  const int s = sums[lane];
  int run = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += y;
  }
  all = __shfl_sync(0xffffffffu, run, 31);
  before = __shfl_sync(0xffffffffu, run - s, warp);
  return before + inc - x;
}

// Which of a thread's kPer pages from page0 on are in use, and how many (past the pool:
// not; the plan's loop over them ends before).
__device__ __forceinline__ int load_used(const PagesParams& p, int page0, bool (&used)[kPer]) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    used[i] = page0 + i < p.num_pages && p.refs[page0 + i] != 0;
    n += used[i];
  }
  return n;
}

// The pages in use of each range.
__global__ void __launch_bounds__(kThreads) fa_pages_count_kernel(const PagesParams p) {
  launch_dependents();
  wait_prior_grid();
  bool used[kPer];
  int all;
  block_scan(load_used(p, (int)blockIdx.x * kPagesRange + (int)threadIdx.x * kPer, used), all);
  if (threadIdx.x == 0) p.range_used[blockIdx.x] = all;
}

// The plan of a fork (kFork) or a compaction: p.to, the free pages in order, p.from,
// the pages copied to them, and how many.
template <bool kFork>
__global__ void __launch_bounds__(kThreads) fa_pages_plan_kernel(const PagesParams p) {
  launch_dependents();
  wait_prior_grid();
  const int tid = threadIdx.x;
  if (kFork && blockIdx.x == (unsigned)p.ranges) {
    // The children, in order.  All parents' lengths are read before the first child
    // is claimed (length -1, until it has its parent's): one that holds keys is
    // nobody's, one that is listed twice that listing's which claims it first.
    const long long cap = (long long)p.max_pages << p.page_shift;
    for (int i = tid; i < p.n; i += kThreads) {
      const int from = p.parents[i], to = p.children[i];
      PagesChild c = {from, to, 0, -1};
      if (from < 0 || from >= p.rows || to < 0 || to >= p.rows || from == to) {
        report(p.status, kSitePagesRow);
        c.child = -1;
      } else {
        c.len = p.seq_lens[from];
        if (c.len < 0 || c.len > cap) {
          report(p.status, kSitePagedLength);
          c.child = -1;
        }
      }
      p.child[i] = c;
    }
    __syncthreads();
    int ranked = 0, all;
    for (int i0 = 0; i0 < p.n; i0 += kThreads) {
      const int i = i0 + tid;
      bool part = false;
      int last = 0;
      if (i < p.n) {
        const PagesChild c = p.child[i];  // (this thread's own)
        if (c.child >= 0) {
          part = (c.len & (p.page_size - 1)) != 0;
          if (part) last = p.page_table[(long long)c.parent * p.max_pages + (c.len >> p.page_shift)];
          if (part && (last < 0 || last >= p.num_pages)) {
            report(p.status, kSitePagedPage);
            p.child[i].child = -1;
            part = false;
          } else if (atomicCAS(p.seq_lens + c.child, 0, -1) != 0) {
            report(p.status, kSitePagesRow);
            p.child[i].child = -1;
            part = false;
          }
        }
      }
      const int rank = ranked + block_scan(part, all);
      ranked += all;
      if (part) {
        p.child[i].rank = rank;
        p.from[rank] = last;
      }
    }
    if (tid == 0) p.counts[0] = ranked;  // pages wanted
    return;
  }
  bool used[kPer];
  const int range = blockIdx.x, page0 = range * kPagesRange + tid * kPer;
  int all, before = 0, live = 0;
  int n = load_used(p, page0, used);
  n = block_scan(n, all);
  if (p.ranges == 1) {
    live = all;
  } else {
    // Of the ranges before this one, and of all.
    for (int r0 = 0; r0 < p.ranges; r0 += kThreads) {
      const int r = r0 + tid, x = r < p.ranges ? p.range_used[r] : 0;
      int sum;
      block_scan(r < range ? x : 0, sum);
      before += sum;
      block_scan(x, sum);
      live += sum;
    }
  }
  int below = before + n;  // pages in use below this thread's next
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int page = page0 + i, holes = page - below;
    if (page >= p.num_pages) break;
    if (!used[i]) {
      if (kFork ? holes < p.n : page < live) p.to[holes] = page;
    } else if (!kFork && page >= live) {
      p.from[live - 1 - below] = page;
      p.rank[page] = live - 1 - below;
    }
    below += used[i];
  }
  if (range == p.ranges - 1) {
    // (Written by the thread of the pool's last page, whose `below` is all.)
    if (page0 < p.num_pages && page0 + kPer >= p.num_pages) {
      p.counts[1] = kFork ? p.num_pages - below : live;  // free pages; pages in use
      if (!kFork && p.live) *p.live = live;
    }
  }
  if (!kFork) {
    // Moves: the free pages below `live`, counted where page `live` lies.
    if (live >= p.num_pages) {
      if (range == 0 && tid == 0) p.counts[0] = 0;
    } else if (live >= page0 && live < page0 + kPer) {
      int at = before + n;
      for (int i = 0; i < live - page0; ++i) at += used[i];
      p.counts[0] = live - at;
    }
  }
}

// Copies pages from[k] to to[k], k < n, in all pools: chunks of up to kChunk bytes,
// dealt to the CTAs in turn.
template <int N>
__device__ __forceinline__ void copy_pages(const PagesParams& p, const PagesPools<N>& pools,
                                           const int* from, const int* to, int n) {
  const long long total = (long long)n * pools.chunks;
  for (long long w = blockIdx.x; w < total; w += gridDim.x) {
    const int k = (int)(w / pools.chunks);
    int chunk = (int)(w - (long long)k * pools.chunks), pool = 0, each;
    char* base = reinterpret_cast<char*>(pools.base[0]);
    unsigned bytes = pools.bytes[0];
    if constexpr (N > 1) {
      int hi = pools.n;  // first[pool] <= chunk < first[hi]
      while (hi - pool > 1) {
        const int mid = (pool + hi) / 2;
        if (pools.first[mid] <= chunk)
          pool = mid;
        else
          hi = mid;
      }
      chunk -= pools.first[pool];
      each = (pool + 1 < pools.n ? pools.first[pool + 1] : pools.chunks) - pools.first[pool];
      base = reinterpret_cast<char*>(pools.base[pool]);
      bytes = pools.bytes[pool];
    } else {
      each = pools.chunks / pools.n;
      pool = chunk / each;
      chunk -= pool * each;
      base += pool * pools.stride;
    }
    // A page's chunks are of one size: [lo, hi) is this one's.
    const unsigned part = ((bytes >> 4) + each - 1) / each << 4;
    const unsigned lo = chunk * part, hi = min(lo + part, bytes);
    const int src = from[k], dst = to[k];
    if (src < 0 || src >= p.num_pages || dst < 0 || dst >= p.num_pages) {
      if (threadIdx.x == 0) report(p.status, kSitePagedPage);
      continue;
    }
    const char* const s = base + (long long)src * bytes;
    char* const d = base + (long long)dst * bytes;
    uint4 x[kCopyEach];
#pragma unroll
    for (int i = 0; i < kCopyEach; ++i) {
      const unsigned at = lo + (i * kCopyThreads + threadIdx.x) * 16;
      if (at < hi) x[i] = *reinterpret_cast<const uint4*>(s + at);
    }
#pragma unroll
    for (int i = 0; i < kCopyEach; ++i) {
      const unsigned at = lo + (i * kCopyThreads + threadIdx.x) * 16;
      if (at < hi) *reinterpret_cast<uint4*>(d + at) = x[i];
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kCopyThreads)
    fa_pages_copy_kernel(const PagesParams p, const __grid_constant__ PagesPools<N> pools) {
  launch_dependents();
  wait_prior_grid();
  copy_pages(p, pools, p.src, p.dst, p.n);
}

// The children's tables, lengths and reference counts, and the copies of their last
// pages.
template <int N>
__global__ void __launch_bounds__(kCopyThreads)
    fa_pages_fork_kernel(const PagesParams p, const __grid_constant__ PagesPools<N> pools) {
  launch_dependents();
  wait_prior_grid();
  const int wanted = p.counts[0], there = p.counts[1];
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const PagesChild c = p.child[i];
    if (c.child < 0) continue;
    if (c.rank >= there) {  // no page is left for it: it stays empty
      if (threadIdx.x == 0) {
        p.seq_lens[c.child] = 0;
        report(p.status, kSitePagesFull);
      }
      continue;
    }
    const int* const from = p.page_table + (long long)c.parent * p.max_pages;
    int* const to = p.page_table + (long long)c.child * p.max_pages;
    const int whole = c.len >> p.page_shift;
    for (int j = threadIdx.x; j < whole; j += kCopyThreads) {
      const int id = from[j];
      to[j] = id;
      if (id >= 0 && id < p.num_pages)
        atomicAdd(p.refs + id, 1);
      else
        report(p.status, kSitePagedPage);
    }
    if (threadIdx.x == 0) {
      if (c.rank >= 0) {
        const int id = p.to[c.rank];
        to[whole] = id;
        p.refs[id] = 1;
      }
      p.seq_lens[c.child] = c.len;
    }
  }
  copy_pages(p, pools, p.from, p.to, min(wanted, there));
}

// One CTA a sequence: its pages count one less, its length is 0.  A row that is
// listed twice is freed once: by the CTA that takes its length.  One of a length out
// of bounds is left as it is.
__global__ void __launch_bounds__(128) fa_pages_free_kernel(const PagesParams p) {
  launch_dependents();
  wait_prior_grid();
  __shared__ int s_len;
  const int row = p.parents[blockIdx.x];
  if (row < 0 || row >= p.rows) {
    if (threadIdx.x == 0) report(p.status, kSitePagesRow);
    return;
  }
  if (threadIdx.x == 0) {
    int len = *static_cast<volatile const int*>(p.seq_lens + row);
    if (len < 0 || len > (long long)p.max_pages << p.page_shift) {
      report(p.status, kSitePagedLength);
      len = 0;
    } else if (len > 0 && atomicCAS(p.seq_lens + row, len, 0) != len) {
      len = 0;
    }
    s_len = len;
  }
  __syncthreads();
  const int len = s_len;
  const int pages = (len + p.page_size - 1) >> p.page_shift;
  const int* const list = p.page_table + (long long)row * p.max_pages;
  for (int j = threadIdx.x; j < pages; j += blockDim.x) {
    const int id = list[j];
    if (id < 0 || id >= p.num_pages) {
      report(p.status, kSitePagedPage);
    } else if (atomicSub(p.refs + id, 1) <= 0) {  // nobody held it
      atomicAdd(p.refs + id, 1);
      report(p.status, kSitePagesRefs);
    }
  }
}

// The moved pages' contents, reference counts and numbers in the tables.
template <int N>
__global__ void __launch_bounds__(kCopyThreads)
    fa_pages_compact_kernel(const PagesParams p, const __grid_constant__ PagesPools<N> pools) {
  launch_dependents();
  wait_prior_grid();
  const int moves = p.counts[0], live = p.counts[1];
  const long long cap = (long long)p.max_pages << p.page_shift;
  for (int k = blockIdx.x * kCopyThreads + threadIdx.x; k < moves; k += gridDim.x * kCopyThreads) {
    const int from = p.from[k], to = p.to[k];
    p.refs[to] = p.refs[from];
    p.refs[from] = 0;
  }
  for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int len = p.seq_lens[row];
    if (len < 0 || len > cap) {
      if (threadIdx.x == 0) report(p.status, kSitePagedLength);
      continue;
    }
    const int pages = (len + p.page_size - 1) >> p.page_shift;
    int* const list = p.page_table + (long long)row * p.max_pages;
    for (int j = threadIdx.x; j < pages; j += kCopyThreads) {
      const int id = list[j];
      if (id < 0 || id >= p.num_pages) {
        report(p.status, kSitePagedPage);
      } else if (id >= live) {
        // (A page that was not counted as held has no place to go to.)
        const int rank = p.rank[id];
        if (rank >= 0 && rank < moves && p.from[rank] == id)
          list[j] = p.to[rank];
        else
          report(p.status, kSitePagesRefs);
      }
    }
  }
  copy_pages(p, pools, p.from, p.to, moves);
}

template <class... Args>
int launch(void (*kernel)(Args...), unsigned grid, unsigned threads, cudaStream_t stream,
           const Args&... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid, 1, 1);
  c.blockDim = dim3(threads, 1, 1);
  c.stream = stream;
  c.attrs = pdl;
  c.numAttrs = 1;
  if (cudaLaunchKernelEx(&c, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

// CTAs for copying up to `pages` pages beside `rows` rows of bookkeeping.
template <int N>
unsigned copy_grid(const PagesPools<N>& pools, long long pages, long long rows, int sm_count) {
  const long long most = (long long)sm_count * (2048 / kCopyThreads);
  const long long want = std::max(pages * pools.chunks, rows);
  return (unsigned)std::max(1ll, std::min(want, most));
}

}  // namespace

int pages_chunks(size_t bytes) { return (int)((bytes + kChunk - 1) / kChunk); }

template <int N>
int launch_pages_copy(const PagesParams& p, const PagesPools<N>& pools, int sm_count,
                      cudaStream_t stream) {
  return launch(fa_pages_copy_kernel<N>, copy_grid(pools, p.n, 0, sm_count), kCopyThreads, stream, p,
                pools);
}

template <int N>
int launch_pages_fork(const PagesParams& p, const PagesPools<N>& pools, int sm_count,
                      cudaStream_t stream) {
  int rc = FA_OK;
  if (p.ranges > 1) rc = launch(fa_pages_count_kernel, p.ranges, kThreads, stream, p);
  if (rc == FA_OK) rc = launch(fa_pages_plan_kernel<true>, p.ranges + 1, kThreads, stream, p);
  if (rc != FA_OK) return rc;
  return launch(fa_pages_fork_kernel<N>, copy_grid(pools, p.n, p.n, sm_count), kCopyThreads, stream, p,
                pools);
}

int launch_pages_free(const PagesParams& p, cudaStream_t stream) {
  return launch(fa_pages_free_kernel, (unsigned)p.n, 128, stream, p);
}

template <int N>
int launch_pages_compact(const PagesParams& p, const PagesPools<N>& pools, int sm_count,
                         cudaStream_t stream) {
  int rc = FA_OK;
  if (p.ranges > 1) rc = launch(fa_pages_count_kernel, p.ranges, kThreads, stream, p);
  if (rc == FA_OK) rc = launch(fa_pages_plan_kernel<false>, p.ranges, kThreads, stream, p);
  if (rc != FA_OK) return rc;
  return launch(fa_pages_compact_kernel<N>, copy_grid(pools, p.num_pages / 2, p.rows, sm_count),
                kCopyThreads, stream, p, pools);
}

#define FA_PAGES_POOLS(N)                                                                       \
  template int launch_pages_copy<N>(const PagesParams&, const PagesPools<N>&, int, cudaStream_t); \
  template int launch_pages_fork<N>(const PagesParams&, const PagesPools<N>&, int, cudaStream_t); \
  template int launch_pages_compact<N>(const PagesParams&, const PagesPools<N>&, int, cudaStream_t);
FA_PAGES_POOLS(1)
FA_PAGES_POOLS(kPagesPools)

}  // namespace fa
