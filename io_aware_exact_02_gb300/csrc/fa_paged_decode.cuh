// fa_paged_decode.cuh -- attention over a paged key/value cache for few query
// rows to a key/value head.  The list of units and its split over the CTAs are
// described in fa_paged.cuh.
//
// Decode kernel.  With a handful of query rows the keys and values are read
// once and used little: the kernel's job is to keep memory busy.  It computes
// the transposed products, so that the 128 keys of a tile, not the few rows,
// fill the tensor core's 128 lanes:
//     S^T [128 keys x N rows] = K [128 x d] Q^T          (N = 16, 32 or 64)
//     O^T [d x N rows]       += V^T [d x 128] P^T [128 x N]
// with K and V exactly as the pages hold them (K-major and MN-major operands).
// A compute thread owns one key: N scores, N exponentials a tile, against 128
// of a row-per-thread layout whose rows would mostly be padding.  The running
// maximum is common to the 128 keys of a tile: a tile whose scores stay within
// kRescaleSlack of it (one vote of the 128 threads) takes no reduction at all,
// each thread keeping the sum of its own keys' probabilities until the unit
// ends.  P goes to shared memory as the B operand of the second product, rounded
// to V's type, as the tensor core multiplies it: that is 0.0015 of the relative
// 0.0023 by which O is off (O's own rounding to bf16 is 0.0017; the row sums are
// those of the unrounded values).
//
// Two compute warpgroups take the units in turn, so that one's ending (sums,
// weights, O out of tensor memory, stores: about 2,500 cycles) runs beside the
// other's tiles; with N = 64 each has half of the columns of every unit
// instead, as a thread's registers hold no more.
//
// Warps: 0-3 and 4-7 compute (and write results), 8 and 10 load K and V (TMA: a
// lane per page box), 9 issues the products, each as soon as its operands are
// there, 11 clears what lies past a unit's keys.
//
// Bound by memory, and by latency where there is little to read.  With 32
// query and 8 key/value heads, d = 128, one row a sequence, the merge included:
// 64 sequences of up to 4K keys in pages of 16 take 101 us (6.1 TB/s of the 6.8
// that a copy reaches), 8 of up to 32K 160 us (6.7 TB/s), one of 1,000 keys
// 10.8 us (5 until its first products, 0.7 a tile, 2.6 for the merge).
// K and V stream through one ring of 32 KB (d = 128) tiles in the order K0 V0
// K1 V1 ..., across units; four S buffers let S run ahead of P V, into the
// next units.
#pragma once

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_softmax.cuh"
#include "sm100_ptx.cuh"

namespace fa {

constexpr int kDecodeRing = 8;  // even: an item's slot belongs to one warpgroup
constexpr int kCompute = 256;  // threads of the compute warps
constexpr int kSBufs = 4;      // S buffers, two for each group
// A row's reference maximum before it has seen a key: finite, so that the
// exponent of a masked score is -inf and not NaN.
constexpr float kNoRef = -3.0e38f;

template <int D, int R>
struct DecodeCfg {
  static constexpr int N = R < 16 ? 16 : R;  // columns of the products
  static constexpr int kTileBytes = kTile * D * 2;
  // As many ring slots as the 227 KB allow beside Q and P; an even number, so
  // that K always takes the even slots and V the odd ones, and the use before
  // in a K tile's slot is a K tile whose S is issued before (in a V tile's, a
  // V tile whose P V is): a barrier is only ever tested for the phase after
  // one that is known to have completed.
  static constexpr int kStages = D == 128 ? (N == 16 ? 6 : 4) : (N == 16 ? 12 : 10);
  static_assert(kStages % 2 == 0, "K and V slots");
  // The warpgroups split a unit's columns (else they take units in turn).
  static constexpr bool kHalves = N == 64;
  // Columns of a thread: of 16, only the 8 that have rows, where that is enough
  // (the others of P stay whatever they are, and of O are not read).
  static constexpr int kCols = kHalves ? N / 2 : R;
  static constexpr uint32_t kTmemCols = 8 * N;  // 4 S buffers, 2 O (a power of two)
  static __device__ __forceinline__ uint32_t col_s(int i) { return (uint32_t)i * N; }
  // O of the units of parity i.
  static __device__ __forceinline__ uint32_t col_o(int i) { return (uint32_t)(kSBufs + i) * N; }
  // The threads that work on a unit together, and their named barrier.
  static constexpr int kGroups = kHalves ? 1 : 2;
  static constexpr int kGroup = kCompute / kGroups;
  // A group's n-th tile uses its S buffer n % 2 and its P buffer n % 2.  S of
  // tile n is issued only after P V of tile n - 2.
  static constexpr int kSPer = 2, kPBufs = 2 * kGroups;
  static __device__ __forceinline__ int barrier(int wg) { return kHalves ? 1 : 2 + wg; }
};

template <int D, int R>
struct alignas(1024) DecodeSmem {
  using Cfg = DecodeCfg<D, R>;
  static constexpr int N = Cfg::N;
  uint8_t kv[Cfg::kStages][Cfg::kTileBytes];
  uint8_t q[2][N * D * 2];       // [d / 64][N rows][128 B], 128B-swizzled
  uint8_t pt[Cfg::kPBufs][N * kTile * 2];  // P: [2 blocks of 64 keys][N rows][128 B], swizzled
  float4 top[2][N];              // column maxima of a warpgroup's four warps
  float sum[2][4][N];            // column sums of a warpgroup's four warps
  float ref[2][N];               // reference maxima of the unit
  float f_own[2][N], f_pre[2][N];  // weights of O and of pre_o
  int lim[2][N];                 // keys row n sees end here
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[Cfg::kStages], kv_empty[Cfg::kStages];
  uint64_t tail_full[Cfg::kStages];  // V tiles with keys past their unit's: loaded, not cleared
  uint64_t s_full[kSBufs], p_full[Cfg::kPBufs], pv_done[Cfg::kPBufs];
  uint64_t o_full[2];
  uint64_t item_full[kDecodeRing], item_empty[kDecodeRing];
  uint64_t drain;
  PagedItem item[kDecodeRing];
  PagedScan scan;
  int of_unit[8];                // the issuing thread's: tiles and item parity of its units
  uint32_t tmem_base;
  int abort_flag;
};

// A vote of `threads` compute threads on named barrier `id`: true for all
// when true for any.  Also a barrier among them.  Every thread of the group
// reaches every vote, failed waits or not: a failure is carried into the next
// vote.
__device__ __forceinline__ bool vote_any(int id, int threads, bool x) {
  int r;
  asm volatile(
      "{\n\t.reg .pred P, Q;\n\t"
      "setp.ne.b32 P, %1, 0;\n\t"
      "barrier.cta.red.or.pred Q, %2, %3, P;\n\t"
      "selp.b32 %0, 1, 0, Q;\n\t}"
      : "=r"(r)
      : "r"((int)x), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

template <int N>
__device__ __forceinline__ void load_cols(uint32_t addr, float (&x)[N]) {
  if constexpr (N == 8) {
    uint32_t r[8];
    tmem_ld8(addr, r);
    tmem_wait_ld8(r);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
  } else if constexpr (N == 16) {
    uint32_t r[16];
    tmem_ld16(addr, r);
    tmem_wait_ld16(r);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
  } else {
    static_assert(N == 32, "columns");
    uint32_t r[32];
    tmem_ld32(addr, r);
    tmem_wait_ld(r);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
  }
}
template <int N>
__device__ __forceinline__ void store_cols(uint32_t addr, const float (&x)[N]) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __float_as_uint(x[i]);
  if constexpr (N == 8)
    tmem_st8(addr, r);
  else if constexpr (N == 16)
    tmem_st16(addr, r);
  else
    tmem_st32(addr, r);
  tmem_wait_st();
}

// Reduces each of N columns (8, 16 or 32) over the warp's 32 lanes, halving the
// columns a lane holds at every step (about N shuffles in all, not 5 N).
// Returns the reduction of column lane / (32 / N).
template <int N, class Op>
__device__ __forceinline__ float reduce_cols(const float (&x)[N], Op op) {
  float y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = x[i];
  const int lane = (int)lane_id();
#pragma unroll
  for (int h = N / 2; h >= 1; h /= 2) {
    const int bit = h * (32 / N);
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float keep = up ? y[i + h] : y[i], send = up ? y[i] : y[i + h];
      y[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, bit));
    }
  }
#pragma unroll
  for (int bit = 16 / N; bit >= 1; bit /= 2) y[0] = op(y[0], __shfl_xor_sync(0xffffffffu, y[0], bit));
  return y[0];
}

// The decode kernel's work on CTA `cta` of the `ctas` that share the phase's
// list.  kStarted: the caller has waited for the prior grid.
template <int D, int R, bool kStarted>
__device__ __forceinline__ void decode_cta(const CUtensorMap* tq, const CUtensorMap* tk,
                                           const CUtensorMap* tv, const PagedParams& p,
                                           const PagedPhase& ph, int cta, int ctas,
                                           uint8_t* smem_raw) {
  using Cfg = DecodeCfg<D, R>;
  constexpr int S = Cfg::kStages, N = Cfg::N, NC = Cfg::kCols;
  constexpr bool kHalves = Cfg::kHalves;
  DecodeSmem<D, R>& sm = *reinterpret_cast<DecodeSmem<D, R>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abortf = &sm.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5;
  constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpLoadV = 10;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&sm.kv_full[s], 1);
      mbar_init(&sm.kv_empty[s], 1);
      mbar_init(&sm.tail_full[s], 1);
    }
    for (int i = 0; i < kSBufs; ++i) mbar_init(&sm.s_full[i], 1);
    for (int i = 0; i < Cfg::kPBufs; ++i) {
      mbar_init(&sm.p_full[i], Cfg::kGroup);
      mbar_init(&sm.pv_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < kDecodeRing; ++i) {
      mbar_init(&sm.item_full[i], 1);
      // Read by the issuing thread, the V and the tail warp, the group's warps.
      mbar_init(&sm.item_empty[i], 3 + Cfg::kGroup / 32);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&sm.tmem_base, Cfg::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kWarpLoad && lane_id() == 0) {
    prefetch_tmap(tq);
    prefetch_tmap(tk);
    prefetch_tmap(tv);
  }
  // Q rows the boxes do not fill (N past the unit's heads) stay zero: their
  // columns of S are never used, and cost nothing as zeros.
  for (int i = tid; i < (int)sizeof(sm.q) / 16; i += kPagedThreads)
    reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  if constexpr (!kStarted) {
    launch_dependents();
    wait_prior_grid();
  }
  PagedWalk walk;
  paged_plan(p, ph, sm.scan, walk, cta, ctas);

  if (warp == kWarpLoad) {
    // ------------------------------------------------------------ Q and K
    setmaxnreg_dec<kPagedRegsLoad>();
    int n_q = 0;  // units loaded
    paged_produce_k<D, S, kDecodeRing>(p, ph, sm, tk, walk, cta, ctas, Cfg::kGroups, [&](const PagedItem& it) {
      const int qb = n_q & 1;
      if (n_q >= 2 && !mbar_wait(&sm.q_empty[qb], ((n_q >> 1) - 1) & 1, p.status, abortf,
                                 kSitePgQEmpty))
        return false;
      if (lane_id() == 0) {
        mbar_arrive_expect_tx(&sm.q_full[qb], ph.tile_tokens * p.G * D * 2);
        for (int h = 0; h < D / 64; ++h)
          tma_load_3d(sm.q[qb] + h * (N * 128), tq, &sm.q_full[qb], h * 64, it.h * p.G, it.tok0);
      }
      ++n_q;
      return true;
    });
    if (*abortf && lane_id() == 0)
      for (int i = n_q - 1; i >= 0 && i >= n_q - 2; --i) drain_wait(&sm.q_full[i & 1], (i >> 1) & 1);
    __syncwarp();
  } else if (warp == kWarpLoadV) {
    // ------------------------------------------------------------ V
    setmaxnreg_dec<kPagedRegsLoad>();
    paged_produce_v<D, S, kDecodeRing>(p, sm, tv, sm.tail_full);
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ products
    setmaxnreg_dec<kPagedRegsLoad>();
    if (lane_id() == 0) {
      const uint32_t id_s = idesc_bf16(128, N, false, false);
      const uint32_t id_o = idesc_bf16(128, N, true, false);
      // The units whose S products are not all issued: the oldest and, if it
      // is the other group's, the next (whose first S can then be issued and
      // worked on before the oldest unit is through).
      struct Cursor {
        int nj, j, tile0, q, u;  // tiles, issued, its first tile, Q use, group; nj = 0: none
      } cur = {0, 0, 0, 0, 0}, nxt = {0, 0, 0, 0, 0};
      int m = 0, units = 0;                // items read, units with keys among them
      int ns[2] = {0, 0}, np[2] = {0, 0};  // S and P V products issued, by group
      int gp = 0;                          // P V products issued
      int p_nj = 0, p_j = 0, p_n = 0;      // the unit of the next P V product
      int ob = 0, p_u = 0;                 // its O, its group
      bool end = false;
      uint32_t idle = 0;
      unsigned long long t0 = 0;
      // S of the cursor's next tile if its K (and Q) has arrived and its
      // buffer's last S has been read (that tile's P V is issued).
      auto try_s = [&](Cursor& k) -> bool {
        if (k.nj == 0 || (k.u ? ns[1] - np[1] : ns[0] - np[0]) >= Cfg::kSPer) return false;
        const int c = 2 * (k.tile0 + k.j), slot = c % S, qb = k.q & 1;
        if (!mbar_test_wait(&sm.kv_full[slot], (c / S) & 1)) return false;
        if (k.j == 0 && !mbar_test_wait(&sm.q_full[qb], (k.q >> 1) & 1)) return false;
        const int sb = k.u * Cfg::kSPer + ((k.u ? ns[1]++ : ns[0]++) & 1);
        tc_fence_after();
        const uint64_t kd = desc_here(sdesc_sw128(smem_u32(sm.kv[slot]), 16, 1024));
        const uint64_t qd = desc_here(sdesc_sw128(smem_u32(sm.q[qb]), 16, 1024));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + Cfg::col_s(sb), desc_plus(kd, (kk >> 2) * (kTile * 128) + (kk & 3) * 32),
                 desc_plus(qd, (kk >> 2) * (N * 128) + (kk & 3) * 32), id_s, kk > 0);
        tc_commit(&sm.s_full[sb]);
        tc_commit(&sm.kv_empty[slot]);
        if (++k.j == k.nj) {
          tc_commit(&sm.q_empty[qb]);
          k.nj = 0;
        }
        return true;
      };
      for (;;) {
        bool did = false;
        // The oldest P V product not issued: P is there, and V.
        if (p_j == p_nj && p_n < units) {
          p_nj = sm.of_unit[p_n & 7] >> 1;
          ob = sm.of_unit[p_n & 7] & 1;
          p_u = kHalves ? 0 : ob;
          p_j = 0;
          ++p_n;
        }
        if (p_j < p_nj) {
          const int n = p_u ? np[1] : np[0], pb = 2 * p_u + (n & 1), c = 2 * gp + 1, slot = c % S;
          if (mbar_test_wait(&sm.p_full[pb], (n >> 1) & 1) &&
              mbar_test_wait(&sm.kv_full[slot], (c / S) & 1)) {
            tc_fence_after();
            // V^T: the tile's 64-channel blocks along M.  At d = 64 there is
            // one block; the product's upper 64 rows repeat the tile 8 keys on
            // and are never read.  The unit's first product overwrites its O,
            // which the group that wrote this P has read for its last unit.
            const uint64_t vd =
                desc_here(sdesc_sw128(smem_u32(sm.kv[slot]), D == 128 ? kTile * 128 : 1024, 1024));
            const uint64_t pd = desc_here(sdesc_sw128(smem_u32(sm.pt[pb]), 16, 1024));
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_ss(tmem + Cfg::col_o(ob), desc_plus(vd, kk * 2048),
                     desc_plus(pd, (kk >> 2) * (N * 128) + (kk & 3) * 32), id_o,
                     (p_j > 0 || kk > 0) ? 1u : 0u);
            tc_commit(&sm.pv_done[pb]);
            tc_commit(&sm.kv_empty[slot]);
            ++gp;
            p_u ? ++np[1] : ++np[0];
            if (++p_j == p_nj) tc_commit(&sm.o_full[ob]);
            did = true;
          }
        } else if (end && cur.nj == 0 && p_n == units) {
          break;
        }
        if (cur.nj == 0) {
          cur = nxt;
          nxt.nj = 0;
        }
        did |= try_s(cur);
        if (nxt.nj > 0) {
          // Ahead of the oldest unit only once that has its Q, and as far as
          // the use before of the tile's slot has had its S issued.
          if (cur.nj == 0 || (nxt.u != cur.u && nxt.q == cur.q + 1 && cur.j > 0 &&
                              nxt.tile0 + nxt.j - S / 2 < cur.tile0 + cur.j))
            did |= try_s(nxt);
        } else if (!end && mbar_test_wait(&sm.item_full[m % kDecodeRing], (m / kDecodeRing) & 1)) {
          // The next segment; one without keys has no products.
          const PagedItem& it = sm.item[m % kDecodeRing];
          end = it.end != 0;
          if (!end && it.nj > 0) {
            nxt.nj = it.nj;
            nxt.j = 0;
            nxt.tile0 = it.tile0;
            nxt.q = units;
            nxt.u = kHalves ? 0 : m & 1;
            sm.of_unit[units & 7] = 2 * it.nj + (m & 1);
            ++units;
          }
          mbar_arrive(&sm.item_empty[m % kDecodeRing]);
          ++m;
          did = true;
        }
        // Nothing was ready: give up after the time limit, or with the CTA.
        if (did) {
          idle = 0;
        } else if ((++idle & 255u) == 0) {
          if (*abortf) break;
          const unsigned long long now = globaltimer_ns();
          if (idle == 256) t0 = now;
          if (now - t0 > kWaitTimeoutNs) {
            report_timeout(p.status, abortf, kSitePgPFull);
            break;
          }
        }
      }
      // Every product issued so far must finish before TMEM is released.
      tc_commit(&sm.drain);
      drain_wait(&sm.drain, 0);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ compute
    setmaxnreg_inc<kPagedRegsCompute>();
    const int wg = warp >> 2, key_t = tid & 127, lane = tid & 31;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float c2 = p.scale_log2, ninf = __int_as_float(0xff800000);
    const int col0 = kHalves ? wg * NC : 0;  // this thread's columns of a unit
    const int buf = kHalves ? 0 : wg;        // its group's copy of the shared arrays
    const int bar = Cfg::barrier(wg);
    const int row = kHalves ? tid : key_t;   // its row of a unit, if below N
    // This thread's place in a row of P: its key's 16-byte chunk (swizzled
    // with the row) and byte in it.
    uint8_t* const pt0 = sm.pt[2 * buf] + (key_t >> 6) * (N * 128) + col0 * 128 + (key_t & 7) * 2;
    const int pchunk = (key_t & 63) >> 3;
    // Row n of a unit is query head n % G of its token n / G.
    const int row_tok = row / p.G, row_head = row % p.G;
    bool fail = false;
    int n_t = 0;             // tiles the group has had
    int n_done[2] = {0, 0};  // units with keys, by the parity of their item
    for (int m = kHalves ? 0 : wg;; m += Cfg::kGroups) {
      PagedItem it;
      it.end = 1;
      it.nj = it.ntok = 0;
      fail = !mbar_wait(&sm.item_full[m % kDecodeRing], (m / kDecodeRing) & 1, p.status, abortf,
                        kSitePgItemFull);
      if (!fail) it = sm.item[m % kDecodeRing];
      __syncwarp();
      if (!fail && lane == 0) mbar_arrive(&sm.item_empty[m % kDecodeRing]);
      const int rows = it.end ? 0 : it.ntok * p.G;
      if (!bound_ok(it.end || (it.tok0 >= 0 && it.tok0 + it.ntok <= p.T && rows <= R && it.h < p.Hkv),
                    p.status, abortf, kChkPgItem))
        fail = true;
      // Keys of the unit's rows (0 for the columns past them).
      if (!fail && !it.end && row < R) {
        int lim = 0;
        if (row < rows) {
          if (ph.whole_batch)
            lim = paged_prefix_limit(p, it.tok0 + row_tok);
          else
            lim = p.causal ? max(0, min(it.pos0 + row_tok + 1, it.len)) : it.len;
        }
        sm.lim[buf][row] = lim;
      }
      if (vote_any(bar, Cfg::kGroup, fail)) break;
      if (it.end) break;
      // Tiles that end at or before min_lim need no masking.
      int min_lim = p.causal ? it.pos0 + 1 : it.len;
      if (ph.whole_batch) {
        min_lim = 0x7fffffff;
        for (int n = 0; n < rows; ++n) min_lim = min(min_lim, sm.lim[buf][n]);
      }
      float ref[NC], l[NC];
      float my_ref = kNoRef;  // thread n < NC: ref[n], for the unit's end
#pragma unroll
      for (int n = 0; n < NC; ++n) ref[n] = kNoRef, l[n] = 0.f;
      const uint32_t colO = tmem + lane_base + Cfg::col_o(m & 1) + col0;
      for (int j = 0; j < it.nj; ++j, ++n_t) {
        const int sb = buf * Cfg::kSPer + n_t % Cfg::kSPer;  // buffers of S, of P
        const int pb = 2 * buf + (n_t & 1);
        const int key = it.key + j * kTile + key_t;
        if (!fail)
          fail = !mbar_wait(&sm.s_full[sb], (n_t / Cfg::kSPer) & 1, p.status, abortf, kSitePgSFull);
        fail = __any_sync(0xffffffffu, fail);  // keep the warp's TMEM accesses converged
        float s[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) s[n] = 0.f;
        if (!fail) {
          tc_fence_after();
          load_cols<NC>(tmem + lane_base + Cfg::col_s(sb) + col0, s);
          tc_fence_before();
        }
        // Exponents before the reference is subtracted; masked: -inf.
        const bool masked = it.key + (j + 1) * kTile > min_lim;
#pragma unroll
        for (int n = 0; n < NC; ++n) s[n] *= c2;
        if (masked) {
#pragma unroll
          for (int n = 0; n < NC; ++n)
            if (key >= sm.lim[buf][col0 + n]) s[n] = ninf;
        }
        float over = s[0] - ref[0];
#pragma unroll
        for (int n = 1; n < NC; ++n) over = fmaxf(over, s[n] - ref[n]);
        // (A unit's first tile has a reference to find in any case.)
        if (j == 0 || vote_any(bar, Cfg::kGroup, over > kRescaleSlack || fail)) {
          // Some score outgrew the reference: move every row's to its maximum.
          const float x = reduce_cols<NC>(s, [](float a, float b) { return fmaxf(a, b); });
          if (lane % (32 / NC) == 0)
            reinterpret_cast<float*>(&sm.top[buf][col0 + lane / (32 / NC)])[warp & 3] = x;
          if (vote_any(bar, Cfg::kGroup, fail)) {
            fail = true;
            break;
          }
          if (key_t < NC) {
            const float4 q = sm.top[buf][col0 + key_t];
            my_ref = fmaxf(fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)), my_ref);
          }
          float alpha[NC];
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const float4 q = sm.top[buf][col0 + n];
            const float top = fmaxf(fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)), ref[n]);
            alpha[n] = ex2_approx(ref[n] - top);
            ref[n] = top;
            l[n] *= alpha[n];
          }
          if (j > 0) {
            // O holds the unit's earlier tiles once their products are done.
            fail = !mbar_wait(&sm.pv_done[pb ^ 1], ((n_t - 1) >> 1) & 1, p.status, abortf,
                              kSitePgPvDone);
            fail = __any_sync(0xffffffffu, fail);
            if (!fail) {
              tc_fence_after();
              float o[NC];
              load_cols<NC>(colO, o);
#pragma unroll
              for (int n = 0; n < NC; ++n) o[n] *= alpha[n];
              store_cols<NC>(colO, o);
              tc_fence_before();
            }
          }
        }
        // P's buffer is free: this S was issued after the product before last,
        // which read it, and products complete in order.
        if (!fail) {
          uint8_t* const pt = pt0 + (n_t & 1) * (N * kTile * 2);
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const float x = ex2_approx(s[n] - ref[n]);
            l[n] += x;
            *reinterpret_cast<__nv_bfloat16*>(pt + n * 128 + ((pchunk ^ (n & 7)) << 4)) =
                __float2bfloat16(x);
          }
          fence_proxy_async_smem();
          mbar_arrive(&sm.p_full[pb]);
        }
      }
      // ------------------------------------------------------ the unit's result
      {
        const float x = reduce_cols<NC>(l, [](float a, float b) { return a + b; });
        if (lane % (32 / NC) == 0) sm.sum[buf][warp & 3][col0 + lane / (32 / NC)] = x;
        if (key_t < NC) sm.ref[buf][col0 + key_t] = my_ref;
      }
      if (vote_any(bar, Cfg::kGroup, fail)) break;
      const bool merge = it.first && ph.pre_o != nullptr;
      if (row < R) {
        const float sum = (sm.sum[buf][0][row] + sm.sum[buf][1][row]) +
                          (sm.sum[buf][2][row] + sm.sum[buf][3][row]);
        float lse2 = sum == 0.f ? ninf : sm.ref[buf][row] + __log2f(sum);
        float own = sum == 0.f ? 0.f : 1.f / sum, pre = 0.f;
        if (row < rows) {
          const long long at = (long long)(it.tok0 + row_tok) * p.Hq + it.h * p.G + row_head;
          if (merge) {
            const float other = ph.pre_lse[at], big = fmaxf(lse2, other);
            if (big != ninf) {
              const float wa = exp2f(lse2 - big), wb = exp2f(other - big), both = wa + wb;
              own *= wa / both;
              pre = wb / both;
              lse2 = big + log2f(both);
            }
          }
          if (it.slot >= 0)
            ph.slot_lse[((long long)cta * 2 + it.slot) * ph.slot_rows + row] = lse2;
          else if (ph.out_lse)
            ph.out_lse[at] = lse2;
          else
            p.lse[at] = lse2 == ninf ? ninf : lse2 * kLn2;
        }
        sm.f_own[buf][row] = own;
        sm.f_pre[buf][row] = pre;
      }
      if (it.nj > 0)
        fail = !mbar_wait(&sm.o_full[m & 1], n_done[m & 1] & 1, p.status, abortf, kSitePgOFull);
      if (vote_any(bar, Cfg::kGroup, fail)) break;
      // O leaves through shared memory, in the group's P buffers (free: the
      // unit's products are done), and is stored eight channels to a thread.
      float* const stage = reinterpret_cast<float*>(sm.pt[2 * buf]);  // [N][D]
      if (it.nj > 0) {
        tc_fence_after();
        float o[NC];
        load_cols<NC>(colO, o);
        tc_fence_before();
        ++n_done[m & 1];
        if (key_t < D) {
#pragma unroll
          for (int n = 0; n < NC; ++n) stage[(col0 + n) * D + key_t] = o[n];
        }
      }
      vote_any(bar, Cfg::kGroup, false);
      for (int i = kHalves ? tid : key_t; i < rows * (D / 8); i += Cfg::kGroup) {
        const int n = i / (D / 8), ch = i % (D / 8) * 8, tok = n / p.G;
        const long long at =
            ((long long)(it.tok0 + tok) * p.Hq + it.h * p.G + (n - tok * p.G)) * D + ch;
        const float f = sm.f_own[buf][n];
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (f != 0.f) {
          x = *reinterpret_cast<const float4*>(stage + n * D + ch);
          y = *reinterpret_cast<const float4*>(stage + n * D + ch + 4);
          x.x *= f, x.y *= f, x.z *= f, x.w *= f;
          y.x *= f, y.y *= f, y.z *= f, y.w *= f;
        }
        const float fp = sm.f_pre[buf][n];
        if (fp != 0.f) {  // only where results are merged in
          const float4 u = *reinterpret_cast<const float4*>(ph.pre_o + at);
          const float4 v = *reinterpret_cast<const float4*>(ph.pre_o + at + 4);
          x.x += fp * u.x, x.y += fp * u.y, x.z += fp * u.z, x.w += fp * u.w;
          y.x += fp * v.x, y.y += fp * v.y, y.z += fp * v.z, y.w += fp * v.w;
        }
        if (it.slot >= 0 || ph.out_o) {
          float* dst = it.slot >= 0
                           ? ph.slot_o +
                                 (((long long)cta * 2 + it.slot) * ph.slot_rows + n) * D + ch
                           : ph.out_o + at;
          reinterpret_cast<float4*>(dst)[0] = x;
          reinterpret_cast<float4*>(dst)[1] = y;
        } else {
          *reinterpret_cast<uint4*>(p.o + at) =
              make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y),
                         pack_bf16x2(y.z, y.w));
        }
      }
      // (The next unit's first vote comes before P is written again.)
    }
  } else {
    // ------------------------------------------------------------ tails
    // Slots past a unit's keys may hold anything, and 0 * NaN is NaN: this
    // warp clears those value rows of a unit's last tile when it has arrived,
    // and hands the tile on.
    setmaxnreg_dec<kPagedRegsLoad>();
    const int lane = (int)lane_id();
    uint32_t parity = 0;  // of tail_full, a bit per slot
    bool ok = true;
    for (int m = 0; ok; ++m) {
      const int is = m % kDecodeRing;
      ok = mbar_wait(&sm.item_full[is], (m / kDecodeRing) & 1, p.status, abortf, kSitePgItemFull);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const PagedItem& it = sm.item[is];
      const int end = it.end, nj = it.nj, slot = (2 * (it.tile0 + nj) - 1) % S;
      const int rows = it.k_hi - (it.key + (nj - 1) * kTile);  // of the last tile
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[is]);
      if (end) break;
      if (nj == 0 || rows >= kTile) continue;
      ok = mbar_wait(&sm.tail_full[slot], (parity >> slot) & 1, p.status, abortf, kSitePgKvFull);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      parity ^= 1u << slot;
      for (int i = rows * 8 + lane; i < kTile * 8; i += 32)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          *reinterpret_cast<uint4*>(sm.kv[slot] + h * (kTile * 128) + i * 16) =
              make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.kv_full[slot]);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

}  // namespace fa
