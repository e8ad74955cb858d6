// fa_pages.h -- the operators on a cache's pages: what the C ABI hands to their
// launchers (fa_pages.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fa {

constexpr int kPagesRange = 4096;  // pages that one CTA scans
constexpr int kPagesPools = 256;   // caches of a call at most

// Sites recorded with FA_ERR_PAGE, after those of the paged cache.
enum : int {
  kSitePagesRow = 305,  // a row number outside the tables, a parent as its own child,
                        // or a child that holds keys
  kSitePagesFull,       // no free page is left for a child
  kSitePagesRefs        // a page that is held but not counted
};

// A fork as planned (child -1: none).
struct PagesChild {
  int parent, child, len;
  int rank;  // of its own page among the free ones, -1: it needs none
};

struct PagesParams {
  const int* parents;   // fork; free: the rows
  const int* children;
  const int* src;       // copy
  const int* dst;
  int* page_table;      // [rows][max_pages]
  int* seq_lens;        // [rows]
  int* refs;            // [num_pages]
  int* live;            // compact: may be null
  int* status;
  int n, rows, max_pages, num_pages, page_size, page_shift, ranges;
  // Workspace: pages used by each range; {copies, free pages or pages in use}; the
  // pages copied, and where to (at most num_pages); fork: the children; compact:
  // a moved page's place in that list.
  int* range_used;
  int* counts;
  int* from;
  int* to;
  PagesChild* child;
  int* rank;
};

// The caches: N = 1, `stride` bytes apart and all alike; else at a base of each.
template <int N>
struct PagesPools {
  int n, chunks;  // chunks: of a page in all of them
  long long stride;
  unsigned long long base[N];
  unsigned bytes[N];  // of a page
  int first[N];       // chunks of the pools before
};
using PagesAlike = PagesPools<1>;
using PagesList = PagesPools<kPagesPools>;

struct PagesWorkspace {
  size_t range_used, counts, from, to, child, rank, total;
};
// n: children, or 0 of a compaction.
inline PagesWorkspace pages_workspace_layout(int num_pages, int n) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  PagesWorkspace w;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up(bytes);
    return here;
  };
  // (Neither more children than forks, nor more moves than half of the pages.)
  const size_t most = n > 0 ? (size_t)n : (size_t)num_pages / 2 + 1;
  w.range_used = take(((size_t)num_pages + kPagesRange - 1) / kPagesRange * sizeof(int));
  w.counts = take(2 * sizeof(int));
  w.from = take(most * sizeof(int));
  w.to = take(most * sizeof(int));
  w.child = take((size_t)n * sizeof(PagesChild));
  w.rank = take(n > 0 ? 0 : (size_t)num_pages * sizeof(int));
  w.total = at;
  return w;
}

// Chunks of a page of so many bytes.
int pages_chunks(size_t bytes);
template <int N>
int launch_pages_copy(const PagesParams& p, const PagesPools<N>& pools, int sm_count,
                      cudaStream_t stream);
template <int N>
int launch_pages_fork(const PagesParams& p, const PagesPools<N>& pools, int sm_count,
                      cudaStream_t stream);
int launch_pages_free(const PagesParams& p, cudaStream_t stream);
template <int N>
int launch_pages_compact(const PagesParams& p, const PagesPools<N>& pools, int sm_count,
                         cudaStream_t stream);

}  // namespace fa
