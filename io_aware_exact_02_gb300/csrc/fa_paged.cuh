// fa_paged.cuh -- what the paged key/value cache kernels share: which
// sequence a packed row belongs to, and the checks of the device-side tables.
//
// The tables (cu_q, seq_lens, page_table) live on the device, so their values
// are checked by the kernels: an entry outside its bounds is recorded as
// FA_ERR_PAGE in the status word, and nothing is read or written through it.
#pragma once

#include "fa_internal.h"
#include "sm100_ptx.cuh"

namespace fa {

// Sites recorded with FA_ERR_PAGE.
enum : int {
  kSitePagedRows = 301,  // cu_q not ascending within [0, T]
  kSitePagedLength,      // a sequence length outside [0, max_pages * page_size]
  kSitePagedPosition,    // a new token's position outside the table (or the rope table)
  kSitePagedPage         // a page number outside [0, num_pages)
};

struct PagedRow {
  int b;    // the row's sequence, -1: none (padding, or bad tables)
  int pos;  // its position in the sequence
};

// The sequence of row t: the largest b with cu_q[b] <= t, found by a
// warp-wide search over 32 probes a step (all lanes of the warp call it with
// the same t).  Rows at and past cu_q[B] belong to none.
__device__ __forceinline__ PagedRow paged_row(const int* cu_q, const int* seq_lens, int B, int T,
                                              int t, int* status) {
  const int lane = (int)lane_id();
  int lo = 0, n = B + 1;  // the answer lies in [lo, lo + n), or before lo = 0
  bool before = true;     // no probe was at or below t yet
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < n && cu_q[i] <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0) break;
    before = false;
    const int last = 31 - __clz((int)m);
    lo += last * step;
    n = min(step, n - last * step);
    if (step == 1) break;
  }
  PagedRow r;
  r.b = -1;
  r.pos = 0;
  if (before || lo >= B) return r;
  const int t0 = cu_q[lo], t1 = cu_q[lo + 1];
  if (t0 > t || t1 <= t || t1 > T) {
    int abort_flag = 0;
    if (lane == 0) report_status(status, &abort_flag, FA_ERR_PAGE, kSitePagedRows);
    return r;
  }
  r.b = lo;
  r.pos = seq_lens[lo] - (t1 - t);
  return r;
}

}  // namespace fa
