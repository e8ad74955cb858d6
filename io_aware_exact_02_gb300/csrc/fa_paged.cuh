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

constexpr float kLn2 = 0.69314718055994530942f;

// Sites recorded with FA_ERR_PAGE.
enum : int {
  kSitePagedRows = 301,  // cu_q not ascending within [0, T]
  kSitePagedLength,      // a sequence length outside [0, max_pages * page_size]
  kSitePagedPosition,    // a new token's position outside the table (or the rope table)
  kSitePagedPage         // a page number outside [0, num_pages)
};
// Wait sites of the paged kernels.
enum : int {
  kSitePgQFull = 311, kSitePgQEmpty, kSitePgKvFull, kSitePgKvEmpty, kSitePgSFull, kSitePgPFull,
  kSitePgPHalf, kSitePgPvDone, kSitePgOFull, kSitePgOEmpty, kSitePgItemFull, kSitePgItemEmpty
};
// Bounds checks of the checked build.
enum : int {
  kChkPgItem = 1301,  // a unit's rows or head
  kChkPgRow,          // an output row
  kChkPgParts         // (in every build) where a row's parts lie, as the join kernel read it
};

struct PagedRow {
  int b;    // the row's sequence, -1: none (padding, or bad tables)
  int pos;  // its position in the sequence
};

// Whether rows t0 .. t1 - 1 can be a sequence's.
__device__ __forceinline__ bool paged_range_ok(int t0, int t1, int T) {
  return t0 >= 0 && t1 >= t0 && t1 <= T;
}

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
  if (t0 > t || t1 <= t || !paged_range_ok(t0, t1, T)) {
    int abort_flag = 0;
    if (lane == 0) report_status(status, &abort_flag, FA_ERR_PAGE, kSitePagedRows);
    return r;
  }
  r.b = lo;
  r.pos = seq_lens[lo] - (t1 - t);
  return r;
}

// ------------------------------------------------------------------ the plan
//
// The work of a call is a list of units: (sequence, key/value head, a run of
// query tokens) in that order, a unit's rows being its tokens' G query heads.
// A unit costs its number of 128-key tiles (one at least), and the list's
// tiles are dealt to the CTAs in equal contiguous ranges, whatever the
// lengths: a CTA's first and last unit may be shared with its neighbours, and
// each of the parts leaves its normalised fp32 O and logsumexp in a slot of
// the workspace (slot 0 of a CTA: its first segment, slot 1: its last) that
// the merge kernel joins in list order; so the result does not depend on
// timing.  Every CTA derives its range from the tables itself: no launch
// needs the lengths on the host.

// Registers of the paged kernels' twelve warps: launched with kPagedRegs a
// thread, of which the third warpgroup (loads, products, one idle warp) hands
// some to the two that compute.  The launchers refuse a kernel compiled with
// fewer, whose setmaxnreg.inc would wait for registers that do not exist.
constexpr int kPagedThreads = 384, kPagedRegs = 168, kPagedRegsCompute = 200, kPagedRegsLoad = 104;
static_assert(2 * 128 * kPagedRegsCompute + 128 * kPagedRegsLoad <= kPagedThreads * kPagedRegs,
              "register split above the launch's total");

// The prompt kernel over the cache in 4 bits has a warpgroup more, which makes the
// tiles: launched with kPaged4Regs a thread.
constexpr int kPaged4Threads = 512, kPaged4Regs = 128, kPaged4RegsCompute = 168,
              kPaged4RegsList = 72, kPaged4RegsTiles = 104;
static_assert(2 * 128 * kPaged4RegsCompute + 128 * (kPaged4RegsList + kPaged4RegsTiles) <=
                  kPaged4Threads * kPaged4Regs,
              "register split above the launch's total");

// Wait without the abort shortcut: used while winding down.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (globaltimer_ns() - t0 > 100000000ull) return;  // 100 ms
  }
}

// The phase of a call a kernel runs.
struct PagedPhase {
  int whole_batch;     // 1: the shared prefix, attended by the rows of the whole batch
  int key0;            // the first key attended (prefix_len after a shared prefix)
  int unit_tokens;     // query tokens of a unit
  int tile_tokens;     // query tokens of a Q tile (decode: the unit's)
  int slot_rows;       // rows of a slot: 8 .. 64, or 256
  int box_out;         // 32 rows of a Q tile are whole tokens, and o is bf16: stored as boxes
  int n_min, n_max;    // sequences of that many new tokens take part
  char* rec;           // PagedRec per CTA
  int* ctas;           // how many CTAs share the phase's list, where not all do; or null
  uint2* parts;        // [T][Hkv], written: paged_parts of the units; or null
  float* slot_o;       // [CTA][2][slot_rows][d]
  float* slot_lse;     // [CTA][2][slot_rows], log2 units
  const float* pre_o;  // results to merge in ([T][Hq][d], [T][Hq], log2 units), or null
  const float* pre_lse;
  float* out_o;        // fp32 results instead of o and lse, or null
  float* out_lse;
};

// What the merge kernel needs to know of a CTA's first unit.
struct PagedRec {
  int split;        // the unit began in an earlier CTA
  int slot, n;      // its first slot, and how many there are: the next CTAs' slots 0 follow
  int tok0, ntok, h;
};
static_assert(sizeof(PagedRec) <= kPagedRecBytes, "record size");

// What the join kernel needs to know of a row's unit: x: its first slot, and
// 2^16 times the number of its slots (1: the whole unit is in out_o); y: where
// the token's rows begin in a slot.  Of a shared prefix's units only the first
// token has one.
__device__ __forceinline__ uint2 paged_parts(int slot, int n, int row) {
  return make_uint2((uint32_t)slot | (uint32_t)n << 16, (uint32_t)row);
}
// Whether n slots from `slot` on, and a row of each, can be what one of `ctas`
// CTAs left: a unit without a word (of a sequence whose tables are out of
// bounds, or of a CTA that gave up on a wait) leaves whatever the workspace
// held, and that is not to be followed out of it.
__host__ __device__ __forceinline__ bool paged_parts_ok(int slot, int n, int row, int ctas,
                                                        int slot_rows) {
  return n >= 1 && slot >= 0 && slot / 2 + n <= ctas && row >= 0 && row < slot_rows;
}

struct PagedSeq {
  int t0, n, len;  // first row, new tokens, keys
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, const PagedPhase& ph, int b) {
  PagedSeq s;
  if (ph.whole_batch) {
    s.t0 = 0;
    s.n = p.T;
    s.len = p.prefix_len;
    return s;
  }
  const int t0 = p.cu_q[b], t1 = p.cu_q[b + 1];
  s.t0 = t0;
  s.n = t1 - t0;
  s.len = p.seq_lens[b];
  int abort_flag = 0;
  if (!paged_range_ok(t0, t1, p.T)) {
    report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedRows);
    s.t0 = s.n = 0;
  }
  if (s.n < ph.n_min || s.n > ph.n_max) s.n = 0;
  if (s.n > 0 && (s.len < 0 || s.len > (p.max_pages << p.page_shift))) {
    report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedLength);
    s.len = s.len < 0 ? 0 : p.max_pages << p.page_shift;
  }
  return s;
}

// Keys [key0, unit_hi) concern the i-th unit of a sequence's head.
__device__ __forceinline__ int paged_unit_hi(const PagedParams& p, const PagedPhase& ph,
                                             const PagedSeq& s, int i) {
  if (ph.whole_batch || !p.causal) return s.len;
  const int e = min((i + 1) * ph.unit_tokens, s.n);
  return max(s.len - s.n + e, 0);
}
__device__ __forceinline__ int paged_unit_tiles(const PagedParams& p, const PagedPhase& ph,
                                                const PagedSeq& s, int i) {
  const int x = paged_unit_hi(p, ph, s, i) - ph.key0;
  return x <= 0 ? 0 : (x + kTile - 1) / kTile;
}
__device__ __forceinline__ int paged_units(const PagedPhase& ph, const PagedSeq& s) {
  return s.n <= ph.unit_tokens ? (s.n > 0) : (s.n + ph.unit_tokens - 1) / ph.unit_tokens;
}
// Groups of the list's split: the units of the whole batch, if each can have a
// CTA, else one.
__device__ __forceinline__ int paged_groups(const PagedParams& p, const PagedPhase& ph, int ctas) {
  if (!ph.whole_batch) return 1;
  const long long units = (long long)p.Hkv * ((p.T + ph.unit_tokens - 1) / ph.unit_tokens);
  return units <= ctas ? (int)units : 1;
}
// Tiles of one head of a sequence.  kEnd: what the end of a unit costs, in tiles;
// the kernels over the cache in 4 bits, whose tiles take less, count it.
template <int kEnd = 0>
__device__ __forceinline__ long long paged_head_cost(const PagedParams& p, const PagedPhase& ph,
                                                     const PagedSeq& s) {
  const int R = paged_units(ph, s);
  if (R == 0) return 0;
  if (!p.causal || ph.whole_batch)
    return (long long)R * (max(1, paged_unit_tiles(p, ph, s, 0)) + kEnd);
  long long c = 0;
  for (int i = 0; i < R; ++i) c += max(1, paged_unit_tiles(p, ph, s, i)) + kEnd;
  return c;
}

// The start of a paged kernel is straight-line code that every launch fetches
// anew, at some 50 ns for eight instructions: what it does more than once is a
// function or a loop here, not inlined copies.

// a / b of nonnegative numbers; nearly always both fit 32 bits, whose division
// is several times shorter.
static __host__ __device__ __noinline__ long long paged_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}

// Two lists side by side: the CTAs, of `ctas` (even, at least 4), that take the
// list of weight wa, the others taking that of weight wb; in proportion to the
// weights, and both multiples of two (whole clusters).  A list with work always
// has a cluster, however little of the whole its work is: a list without CTAs
// would leave its rows unwritten.  groups (at most ctas - 2): the units of the
// first list that are dealt whole (PagedShare), whose CTAs are a multiple of
// them before they are made even.
__host__ __device__ __forceinline__ int paged_duo_split(long long wa, long long wb, int ctas,
                                                        int groups) {
  if (wa <= 0) return 0;
  if (wb <= 0) return ctas;
  int na = (int)paged_div(wa * ctas + (wa + wb) / 2, wa + wb);
  na = (na + groups / 2) / groups * groups;
  if (na < groups) na = groups;
  if (na > ctas - 2) na -= groups;
  na = (na + 1) & ~1;
  return na < ctas - 2 ? na : ctas - 2;
}

// CTA c's range of the list is [lo(c), lo(c + 1)): equal ranges, the first
// `more` of them one tile longer; with fewer tiles than CTAs the first ones
// take one each.  A list of `groups` units of equal cost, no more than there
// are CTAs, is dealt unit by unit to as many CTAs each, so that no CTA has
// parts of two (a second segment costs a prompt CTA 10 us and more).
struct PagedShare {
  long long total, per, each;  // tiles: in all, of a group, of a CTA
  int k, more;                 // CTAs of a group
  PagedShare() = default;
  __device__ __forceinline__ PagedShare(long long t, int ctas, int groups) : total(t) {
    per = groups > 1 ? paged_div(t, groups) : t;
    k = groups > 1 ? ctas / groups : ctas;
    each = paged_div(per, k);
    more = (int)(per - each * k);
  }
  __device__ __forceinline__ long long lo(int c) const {
    const int g = per == total ? 0 : c / k, r = c - g * k;
    const long long x = g * per + each * r + (r < more ? r : more);
    return x < total ? x : total;
  }
  // The CTA whose range holds tile x of the list.
  __device__ __forceinline__ int owner(long long x) const {
    const int g = per == total ? 0 : (int)paged_div(x, per);
    x -= g * per;
    const long long head = (each + 1) * more;
    return g * k + (x < head ? (int)paged_div(x, each + 1) : more + (int)paged_div(x - head, each));
  }
};

// One segment of a unit, as the producer hands it to the other roles.
struct PagedItem {
  int end;        // 1: no more items
  int nj;         // key tiles (0: the unit has no keys)
  int b, h;
  int tok0, ntok; // the unit's rows: packed rows tok0 .. tok0 + ntok - 1
  int key;        // the segment's first key
  int k_hi;       // the unit's keys end here
  int pos0;       // row tok0's position (whole_batch: unused)
  int len;
  int slot;       // -1: the whole unit, written straight to the output; else 0 or 1
  int first;      // the segment begins the unit (and merges pre_o in)
  int tile0;      // key tiles of the CTA's segments before this one
};

// A CTA's walk along its range of the list.
struct PagedWalk {
  long long g, hi;
  long long start, end;  // of the last segment's unit, in the list
  PagedShare share;
  int b, h, i, tile, units, tiles;
  PagedSeq s;
  bool first;
};

struct PagedScan {
  long long warp_sum[32];
  long long excl, head;  // of the sequence that holds the CTA's first tile
  PagedSeq s;
  int b;
};

// The cost of sequence b (0 past the last), and of one of its heads.
template <int kEnd = 0>
__device__ __forceinline__ long long paged_cost(const PagedParams& p, const PagedPhase& ph, int b,
                                                int B, PagedSeq& s, long long& head) {
  head = 0;
  if (b < B) {
    s = paged_seq(p, ph, b);
    head = paged_head_cost<kEnd>(p, ph, s);
  }
  return head * p.Hkv;
}
__device__ __forceinline__ long long warp_scan(long long x) {  // inclusive
  const int lane = (int)lane_id();
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The list's length and the sequence that holds the CTA's first tile.  Up to
// 32 sequences are left to the K warp alone (paged_walk_begin), a lane each.
// More take all threads of the CTA: one scan of the sequences' costs where a
// thread has one at most, else a sum and a second pass.
template <int kEnd = 0>
__device__ __forceinline__ void paged_plan(const PagedParams& p, const PagedPhase& ph,
                                           PagedScan& sc, PagedWalk& w, int cta, int ctas) {
  const int B = ph.whole_batch ? 1 : p.B;
  if (B <= 32) return;
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, nw = nt >> 5;
  PagedSeq s;
  long long head;
  // The sum of the costs of the warps before this one's and of all.
  auto sums = [&](long long of_warp, long long& before, long long& all) {
    if (lane == 31) sc.warp_sum[warp] = of_warp;
    __syncthreads();
    before = all = 0;
    for (int i = 0; i < nw; ++i) {
      if (i < warp) before += sc.warp_sum[i];
      all += sc.warp_sum[i];
    }
  };
  long long total = 0, before, all, inc = 0;
  if (B > nt) {
    for (int b = tid; b < B; b += nt) inc += paged_cost<kEnd>(p, ph, b, B, s, head);
    sums(warp_scan(inc), before, total);
    __syncthreads();
  }
  long long run = 0;
  for (int b0 = 0; b0 < B; b0 += nt) {
    const long long cost = paged_cost<kEnd>(p, ph, b0 + tid, B, s, head);
    inc = warp_scan(cost);
    sums(inc, before, all);
    if (B <= nt) total = all;
    w.share = PagedShare(total, ctas, 1);
    w.g = w.share.lo(cta);
    w.hi = w.share.lo(cta + 1);
    const long long excl = run + before + inc - cost;
    if (cost > 0 && excl <= w.g && w.g < excl + cost) {
      sc.b = b0 + tid;
      sc.excl = excl;
      sc.head = head;
      sc.s = s;
    }
    run += all;
    __syncthreads();
    if (w.g < run) break;  // found
  }
}

// The work in two phases' lists, tiles times the one weight and units times the
// other, by every warp for itself.
struct PagedWeight {
  int tile, unit;
};
__device__ __forceinline__ void paged_weights(const PagedParams& p, const PagedPhase& pa,
                                              PagedWeight a, const PagedPhase& pb, PagedWeight b,
                                              long long& wa, long long& wb) {
  auto weigh = [&](const PagedPhase& ph, PagedWeight w, int i) -> long long {
    const PagedSeq s = paged_seq(p, ph, i);
    return (paged_head_cost(p, ph, s) * w.tile + (long long)paged_units(ph, s) * w.unit) * p.Hkv;
  };
  wa = wb = 0;
  for (int i = (int)lane_id(); i < p.B; i += 32) {
    if (!pa.whole_batch) wa += weigh(pa, a, i);
    wb += weigh(pb, b, i);
  }
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    wa += __shfl_xor_sync(0xffffffffu, wa, o);
    wb += __shfl_xor_sync(0xffffffffu, wb, o);
  }
  if (pa.whole_batch) wa = weigh(pa, a, 0);
}

// The K warp's start of the walk.
template <int kEnd = 0>
__device__ __forceinline__ void paged_walk_begin(const PagedParams& p, const PagedPhase& ph,
                                                 const PagedScan& sc, PagedWalk& w, int cta,
                                                 int ctas) {
  w.first = true;
  w.tiles = 0;
  const int B = ph.whole_batch ? 1 : p.B;
  long long head, off;
  if (B <= 32) {
    const long long cost = paged_cost<kEnd>(p, ph, (int)lane_id(), B, w.s, head);
    const long long inc = warp_scan(cost);
    w.share = PagedShare(__shfl_sync(0xffffffffu, inc, 31), ctas, paged_groups(p, ph, ctas));
    w.g = w.share.lo(cta);
    w.hi = w.share.lo(cta + 1);
    if (w.g >= w.hi) return;  // idle CTA
    const unsigned at = __ballot_sync(0xffffffffu, inc - cost <= w.g && w.g < inc);
    w.b = __ffs((int)at) - 1;
    w.s.t0 = __shfl_sync(0xffffffffu, w.s.t0, w.b);
    w.s.n = __shfl_sync(0xffffffffu, w.s.n, w.b);
    w.s.len = __shfl_sync(0xffffffffu, w.s.len, w.b);
    head = __shfl_sync(0xffffffffu, head, w.b);
    off = w.g - __shfl_sync(0xffffffffu, inc - cost, w.b);
  } else {
    if (w.g >= w.hi) return;  // idle CTA
    w.b = sc.b;
    w.s = sc.s;
    head = sc.head;
    off = w.g - sc.excl;
  }
  w.units = paged_units(ph, w.s);
  w.h = (int)paged_div(off, head);
  off -= w.h * head;
  w.i = 0;
  if (!p.causal || ph.whole_batch) {  // units of equal cost
    const int c = max(1, paged_unit_tiles(p, ph, w.s, 0)) + kEnd;
    w.i = (int)paged_div(off, c);
    off -= (long long)w.i * c;
  } else {
    for (;; ++w.i) {
      const int c = max(1, paged_unit_tiles(p, ph, w.s, w.i)) + kEnd;
      if (off < c) break;
      off -= c;
    }
  }
  w.tile = (int)off;
}

// The walk's next segment.
__device__ __forceinline__ PagedItem paged_next(const PagedParams& p, const PagedPhase& ph,
                                                PagedWalk& w, int cta) {
  PagedItem it = {};
  it.end = w.g >= w.hi ? 1 : 0;
  if (it.end) return it;
  const int tiles = paged_unit_tiles(p, ph, w.s, w.i), cost = max(1, tiles);
  const int take = (int)min((long long)(cost - w.tile), w.hi - w.g);
  it.nj = tiles == 0 ? 0 : take;
  it.b = w.b;
  it.h = w.h;
  it.tok0 = w.s.t0 + w.i * ph.unit_tokens;
  it.ntok = min(ph.unit_tokens, w.s.n - w.i * ph.unit_tokens);
  it.key = ph.key0 + w.tile * kTile;
  it.k_hi = paged_unit_hi(p, ph, w.s, w.i);
  it.pos0 = w.s.len - w.s.n + w.i * ph.unit_tokens;
  it.len = w.s.len;
  it.slot = take == cost ? -1 : (w.first ? 0 : 1);
  it.first = w.tile == 0;
  it.tile0 = w.tiles;
  w.tiles += it.nj;
  w.start = w.g - w.tile;
  w.end = w.start + cost;
  w.first = false;
  w.g += take;
  w.tile += take;
  if (w.tile == cost && w.g < w.hi) {
    w.tile = 0;
    if (++w.i == w.units) {
      w.i = 0;
      if (++w.h == p.Hkv) {
        w.h = 0;
        do {  // the range's end bounds the walk: a later sequence has tiles
          ++w.b;
          w.s = paged_seq(p, ph, w.b);
        } while (w.s.n == 0 && w.b + 1 < p.B);
        w.units = paged_units(ph, w.s);
      }
    }
  }
  return it;
}

// The same where a unit's end counts as kEnd tiles, which lie behind the unit's
// own: a range that has none but such of a unit has no segment of it.
template <int kEnd>
__device__ __forceinline__ PagedItem paged_next_weighed(const PagedParams& p, const PagedPhase& ph,
                                                        PagedWalk& w, int cta) {
  PagedItem it = {};
  for (;;) {
    it.end = w.g >= w.hi ? 1 : 0;
    if (it.end) return it;
    const int tiles = paged_unit_tiles(p, ph, w.s, w.i), real = max(1, tiles), cost = real + kEnd;
    const int take = (int)min((long long)(cost - w.tile), w.hi - w.g);
    const int own = min(w.tile + take, real) - w.tile;
    if (own > 0) {
      it.nj = tiles == 0 ? 0 : own;
      it.b = w.b;
      it.h = w.h;
      it.tok0 = w.s.t0 + w.i * ph.unit_tokens;
      it.ntok = min(ph.unit_tokens, w.s.n - w.i * ph.unit_tokens);
      it.key = ph.key0 + w.tile * kTile;
      it.k_hi = paged_unit_hi(p, ph, w.s, w.i);
      it.pos0 = w.s.len - w.s.n + w.i * ph.unit_tokens;
      it.len = w.s.len;
      it.first = w.tile == 0;
      it.tile0 = w.tiles;
      w.tiles += it.nj;
      w.start = w.g - w.tile;
      w.end = w.start + real;
      it.slot = own == real ? -1 : (w.start > w.share.lo(cta) ? 1 : 0);
    }
    w.first = false;
    w.g += take;
    w.tile += take;
    if (w.tile == cost && w.g < w.hi) {
      w.tile = 0;
      if (++w.i == w.units) {
        w.i = 0;
        if (++w.h == p.Hkv) {
          w.h = 0;
          do {  // the range's end bounds the walk: a later sequence has tiles
            ++w.b;
            w.s = paged_seq(p, ph, w.b);
          } while (w.s.n == 0 && w.b + 1 < p.B);
          w.units = paged_units(ph, w.s);
        }
      }
    }
    if (own > 0) return it;
  }
}

// What the merge needs to know of a CTA's first unit, `it` being its first segment,
// the walk's last.
__device__ __forceinline__ PagedRec paged4_first_rec(const PagedItem& it, const PagedWalk& w) {
  PagedRec r = {};  // (a CTA whose first segment begins its unit joins none)
  if (!it.first) {
    const int c0 = w.share.owner(w.start);
    r.split = 1;
    r.slot = 2 * c0 + (w.share.lo(c0) < w.start ? 1 : 0);
    r.n = w.share.owner(w.end - 1) - c0 + 1;
    r.tok0 = it.tok0;
    r.ntok = it.ntok;
    r.h = it.h;
  }
  return r;
}

// Keys row t of the batch sees of the shared prefix.
__device__ __forceinline__ int paged_prefix_limit(const PagedParams& p, int t) {
  if (t >= p.T) return 0;
  // The largest b with cu_q[b] <= t, b = t first: one token per sequence.
  const int g = min(t, p.B - 1);
  const int first = p.cu_q[0], end = p.cu_q[p.B], at = p.cu_q[g], after = p.cu_q[g + 1];
  if (first > t || end <= t) return 0;  // a padding row
  int lo = 0, hi = p.B;  // cu_q[lo] <= t < cu_q[hi]
  if (at <= t) lo = g;
  if (after > t) hi = g + 1;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (p.cu_q[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int len = p.seq_lens[lo];
  const int lim = p.causal ? len - (p.cu_q[lo + 1] - t) + 1 : len;
  return max(0, min(lim, p.prefix_len));
}

// The page numbers of a segment, 32 at a time in the lanes of a producer warp,
// the next 32 in flight while these are used.
struct PagedPages {
  const int* list;  // the sequence's page numbers
  int n;            // pages of the unit's keys end here
  int base, cur, next;
};
__device__ __forceinline__ int paged_page_at(const PagedParams& p, const PagedPages& g, int i) {
  if (i >= g.n) return -1;  // past the unit's keys: read as zeros
  return i < (p.prefix_len >> p.page_shift) ? p.prefix_pages[i] : g.list[i];
}
__device__ __forceinline__ void paged_pages_begin(const PagedParams& p, const PagedItem& it,
                                                  PagedPages& g) {
  g.list = p.page_table + (long long)it.b * p.max_pages;
  g.n = it.nj == 0 ? 0 : (it.k_hi + p.page_size - 1) >> p.page_shift;
  g.base = it.key >> p.page_shift;
  g.cur = paged_page_at(p, g, g.base + (int)lane_id());
  g.next = paged_page_at(p, g, g.base + 32 + (int)lane_id());
}

// A producer warp's loads of one 128-key tile of K (or V): one box per page
// (at most 128 rows) and 64 channels, a lane to a box.  A box takes the warp
// about 70 cycles to issue, 16 of them (pages of 16 keys, d = 128) half of the
// time in which a tile arrives: K and V have a warp each.
struct PagedBox {
  bool on;       // the lane has a box
  int sub;       // its page among the tile's
  int x;         // its first channel
  int dst;       // its place in the tile, bytes
  int in_page;   // bits of the key that give its first row in the page
};
template <int D>
__device__ __forceinline__ PagedBox paged_box(const PagedParams& p) {
  const int lane = (int)lane_id(), rows = min(p.page_size, kTile);
  const int shift = max(7 - p.page_shift, 0);  // log2 of the tile's pages
  const int half = lane >> shift;
  PagedBox b;
  b.on = half < D / 64;
  b.sub = lane & ((1 << shift) - 1);
  b.x = half * 64;
  b.dst = half * (kTile * 128) + b.sub * rows * 128;
  b.in_page = (p.page_size - 1) & ~(rows - 1);
  return b;
}
template <int D>
__device__ __forceinline__ void paged_load_tile(const PagedParams& p, const PagedBox& box,
                                                const CUtensorMap* map, PagedPages& g, int h,
                                                int key, uint8_t* dst, uint64_t* bar) {
  const int first = key >> p.page_shift;
  // A tile's pages are a power of two in number, and runs of them start with
  // the segment's first page: they never straddle the 32 at hand.
  if (first >= g.base + 32) {
    g.base += 32;
    g.cur = g.next;
    g.next = paged_page_at(p, g, g.base + 32 + (int)lane_id());
  }
  int id = __shfl_sync(0xffffffffu, g.cur, (first + box.sub - g.base) & 31);
  if (lane_id() == 0) mbar_arrive_expect_tx(bar, kTile * D * 2);
  __syncwarp();
  if (box.on) {
    if (id < 0 || id >= p.num_pages) {
      // Past the unit's keys, or no page: read as zeros, from past the map.
      int abort_flag = 0;
      if (first + box.sub < g.n) report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPage);
      id = p.num_pages;
    }
    tma_load_3d(dst + box.dst, map, bar, box.x, key & box.in_page,
                id * p.Hkv + (id == p.num_pages ? 0 : h));
  }
}

// The two producer warps of a paged kernel.  The K warp walks the CTA's range
// of the list, publishes the segments in the item ring (kRing slots), each as
// soon as the one before has its first tile on the way, loads Q (load_q) and
// K; the V warp follows the ring.  K and V tiles take the slots of the K/V
// ring (S of them, tile_bytes each) in turn.  `ends` records end the list.
template <int D, int S, int kRing, class Smem, class LoadQ>
__device__ __forceinline__ void paged_produce_k(const PagedParams& p, const PagedPhase& ph,
                                                Smem& sm, const CUtensorMap* tk, PagedWalk& walk,
                                                int cta, int ctas, int ends, LoadQ&& load_q) {
  volatile int* abortf = &sm.abort_flag;
  const int lane = (int)lane_id();
  const PagedBox box = paged_box<D>(p);
  bool ok = true;
  int c = 0;  // ring uses
  // Publishes the walk's next segment as item m; false at the list's end (or
  // after a failed wait).  Only this warp writes the records, so it can read
  // them again later.
  auto publish = [&](int m) -> bool {
    const PagedItem it = paged_next(p, ph, walk, cta);
    const int is = m % kRing;
    if (m >= kRing)
      ok = mbar_wait(&sm.item_empty[is], (m / kRing - 1) & 1, p.status, abortf, kSitePgItemEmpty);
    ok = __all_sync(0xffffffffu, ok);
    if (ok && lane == 0) {
      sm.item[is] = it;
      mbar_arrive(&sm.item_full[is]);
    }
    __syncwarp();
    return ok && !it.end;
  };
  paged_walk_begin(p, ph, sm.scan, walk, cta, ctas);
  // What the kernels that join parts need to know, once the segment's loads
  // are on the way: of the CTA's first unit, and of a unit that begins here.
  auto describe = [&](const PagedItem& it, bool first) {
    const bool begins = it.first != 0;
    if (first && begins && lane == 0) reinterpret_cast<PagedRec*>(ph.rec + cta * kPagedRecBytes)->split = 0;
    if (begins ? ph.parts == nullptr : !first) return;
    int c0 = cta, n = 1;
    if (it.slot >= 0) {
      if (!begins) c0 = walk.share.owner(walk.start);
      n = walk.share.owner(walk.end - 1) - c0 + 1;
    }
    if (!begins) {
      PagedRec r;
      r.split = 1;
      r.slot = 2 * c0 + (walk.share.lo(c0) < walk.start ? 1 : 0);
      r.n = n;
      r.tok0 = it.tok0;
      r.ntok = it.ntok;
      r.h = it.h;
      if (lane == 0) *reinterpret_cast<PagedRec*>(ph.rec + cta * kPagedRecBytes) = r;
    } else if (lane < (ph.whole_batch ? 1 : it.ntok)) {
      ph.parts[(long long)(it.tok0 + lane) * p.Hkv + it.h] =
          paged_parts(2 * cta + max(it.slot, 0), n, lane * p.G);
    }
  };
  if (walk.g >= walk.hi && lane == 0)
    reinterpret_cast<PagedRec*>(ph.rec + cta * kPagedRecBytes)->split = 0;
  PagedPages pages, after;
  int m = 0;
  bool more = publish(0);
  if (more) paged_pages_begin(p, sm.item[0], pages);
  for (; more; ++m) {
    const int nj = sm.item[m % kRing].nj, h = sm.item[m % kRing].h;
    int key = sm.item[m % kRing].key;
    auto look_ahead = [&] {
      describe(sm.item[m % kRing], m == 0);
      more = publish(m + 1);
      if (more) paged_pages_begin(p, sm.item[(m + 1) % kRing], after);
    };
    if (nj == 0) {
      look_ahead();
    } else {
      ok = load_q(sm.item[m % kRing]);
      ok = __all_sync(0xffffffffu, ok);
    }
    for (int j = 0; j < nj && ok; ++j, c += 2, key += kTile) {
      const int slot = c % S;
      if (c >= S)
        ok = mbar_wait(&sm.kv_empty[slot], (c / S - 1) & 1, p.status, abortf, kSitePgKvEmpty);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      paged_load_tile<D>(p, box, tk, pages, h, key, sm.kv[slot], &sm.kv_full[slot]);
      if (j == 0) look_ahead();
    }
    if (!ok) break;
    pages = after;
  }
  // Item m is the first end.
  for (int e = 1; e < ends && ok; ++e) publish(m + e);
  if (!ok && lane == 0) {
    // Let the copies already issued land before the CTA exits.
    for (int cc = c - 2; cc >= 0 && cc > c - 2 - S; cc -= 2)
      drain_wait(&sm.kv_full[cc % S], (cc / S) & 1);
  }
  __syncwarp();
}

// tail: the barriers (one per slot) of tiles that reach past their unit's keys,
// or null: such tiles are no different.
template <int D, int S, int kRing, class Smem>
__device__ __forceinline__ void paged_produce_v(const PagedParams& p, Smem& sm,
                                                const CUtensorMap* tv, uint64_t* tail) {
  volatile int* abortf = &sm.abort_flag;
  const int lane = (int)lane_id();
  const PagedBox box = paged_box<D>(p);
  bool ok = true;
  int c = 1;
  // Takes item m if it has been published (or: waits for it).
  int nj, h, key, hi, end, nj2, h2, key2, hi2, end2 = 1;
  PagedPages pages, after;
  uint32_t on_tail = 0;  // slots whose last use completes on tail's barrier
  auto take = [&](int m, bool wait, int& nj, int& h, int& key, int& hi, int& end,
                  PagedPages& pages) -> bool {
    const int is = m % kRing;
    bool there = mbar_test_wait(&sm.item_full[is], (m / kRing) & 1);
    if (!there && wait) {
      ok = mbar_wait(&sm.item_full[is], (m / kRing) & 1, p.status, abortf, kSitePgItemFull);
      there = ok;
    }
    there = __all_sync(0xffffffffu, there);
    ok = __all_sync(0xffffffffu, ok);
    if (!there) return false;
    const PagedItem& it = sm.item[is];
    nj = it.nj, h = it.h, key = it.key, hi = it.k_hi, end = it.end;
    if (!end) paged_pages_begin(p, it, pages);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[is]);
    return true;
  };
  end = 1;
  take(0, true, nj, h, key, hi, end, pages);
  for (int m = 0; ok && !end; ++m) {
    bool have = false;
    for (int j = 0; j < nj && ok; ++j, c += 2, key += kTile) {
      const int slot = c % S;
      if (c >= S)
        ok = mbar_wait(&sm.kv_empty[slot], (c / S - 1) & 1, p.status, abortf, kSitePgKvEmpty);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const bool last = tail != nullptr && key + kTile > hi;
      on_tail = (on_tail & ~(1u << slot)) | ((uint32_t)last << slot);
      paged_load_tile<D>(p, box, tv, pages, h, key, sm.kv[slot],
                         last ? &tail[slot] : &sm.kv_full[slot]);
      if (!have) have = take(m + 1, false, nj2, h2, key2, hi2, end2, after);
    }
    if (ok && !have) take(m + 1, true, nj2, h2, key2, hi2, end2, after);
    if (!ok) break;
    nj = nj2, h = h2, key = key2, hi = hi2, end = end2;
    pages = after;
  }
  if (!ok && lane == 0) {
    for (int cc = c - 2; cc >= 0 && cc > c - 2 - S; cc -= 2) {
      const int slot = cc % S;
      if ((on_tail >> slot) & 1) {
        // Its phase is not counted here: whichever is under way ends.
        drain_wait(&tail[slot], 0);
        drain_wait(&tail[slot], 1);
      } else {
        drain_wait(&sm.kv_full[slot], (cc / S) & 1);
      }
    }
  }
  __syncwarp();
}

}  // namespace fa
