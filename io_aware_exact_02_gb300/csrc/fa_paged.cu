// fa_paged.cu -- attention over a paged key/value cache on sm_103a: the decode
// kernel (few query rows to a key/value head) and the merge of split units;
// fa_paged_prompt.cu holds the kernel for many rows.  The list of units both
// kernels share is described in fa_paged.cuh.
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
// ends.  P goes to shared memory as the B operand of the second product.
//
// Warps: 0-3 compute (and write results), 4 producer (TMA: a lane per page
// box), 5 issues the products.  K and V stream through one ring of 32 KB (d =
// 128) tiles in the order K0 V0 K1 V1 ..., across units; S and P have two
// buffers and O one per unit parity, so that the next tile's (and the next
// unit's) S is there before this one's P is done.
#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_paged_launch.h"
#include "fa_softmax.cuh"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kItemRing = 4;
constexpr int kDecodeThreads = 192;
constexpr int kCompute = 128;  // threads of the compute warps

template <int D, int N>
struct DecodeCfg {
  static constexpr int kTileBytes = kTile * D * 2;
  // As many ring slots as the 227 KB allow beside Q and P.
  static constexpr int kStages =
      D == 128 ? (N == 16 ? 6 : (N == 32 ? 5 : 4)) : (N == 64 ? 10 : 12);
  static constexpr uint32_t kTmemCols = 4 * N;  // S twice, O twice
  static __device__ __forceinline__ uint32_t col_s(int i) { return (uint32_t)i * N; }
  static __device__ __forceinline__ uint32_t col_o(int i) { return (uint32_t)(2 + i) * N; }
};

template <int D, int N>
struct alignas(1024) DecodeSmem {
  uint8_t kv[DecodeCfg<D, N>::kStages][DecodeCfg<D, N>::kTileBytes];
  uint8_t q[2][N * D * 2];    // [d / 64][N rows][128 B], 128B-swizzled
  uint8_t pt[2][N * kTile * 2];  // P: [2 blocks of 64 keys][N rows][128 B], swizzled
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[DecodeCfg<D, N>::kStages], kv_empty[DecodeCfg<D, N>::kStages];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t o_full[2], o_empty[2];
  uint64_t item_full[kItemRing], item_empty[kItemRing];
  uint64_t drain;
  PagedItem item[kItemRing];
  PagedScan scan;
  int lim[N];            // keys row n sees end here
  float top[4][N];       // per compute warp: a tile's column maxima
  float sum[4][N];       // and the unit's column sums
  float f_own[N], f_pre[N], lse2[N];
  uint32_t tmem_base;
  int abort_flag;
};

// Wait without the abort shortcut: used while winding down.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (globaltimer_ns() - t0 > 100000000ull) return;  // 100 ms
  }
}

// A vote of the 128 compute threads: true for all when true for any.  Also a
// barrier among them.  Every compute thread reaches every vote, failed waits
// or not: a failure is carried into the next vote.
__device__ __forceinline__ bool compute_any(bool x) {
  int r;
  asm volatile(
      "{\n\t.reg .pred P, Q;\n\t"
      "setp.ne.b32 P, %1, 0;\n\t"
      "barrier.cta.red.or.pred Q, 1, 128, P;\n\t"
      "selp.b32 %0, 1, 0, Q;\n\t}"
      : "=r"(r)
      : "r"((int)x)
      : "memory");
  return r != 0;
}

template <int N>
__device__ __forceinline__ void load_cols(uint32_t addr, float (&x)[N]) {
  if constexpr (N == 16) {
    uint32_t r[16];
    tmem_ld16(addr, r);
    tmem_wait_ld16(r);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
  } else {
#pragma unroll
    for (int c = 0; c < N / 32; ++c) {
      uint32_t r[32];
      tmem_ld32(addr + c * 32, r);
      tmem_wait_ld(r);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[c * 32 + i] = __uint_as_float(r[i]);
    }
  }
}
template <int N>
__device__ __forceinline__ void store_cols(uint32_t addr, const float (&x)[N]) {
  if constexpr (N == 16) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(x[i]);
    tmem_st16(addr, r);
  } else {
#pragma unroll
    for (int c = 0; c < N / 32; ++c) {
      uint32_t r[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(x[c * 32 + i]);
      tmem_st32(addr + c * 32, r);
    }
  }
  tmem_wait_st();
}

template <int D, int N>
__global__ void __launch_bounds__(kDecodeThreads, 1)
    fa_paged_decode_kernel(const __grid_constant__ CUtensorMap tq,
                           const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv, const PagedParams p,
                           const PagedPhase ph) {
  using Cfg = DecodeCfg<D, N>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  DecodeSmem<D, N>& sm = *reinterpret_cast<DecodeSmem<D, N>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abortf = &sm.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5;
  constexpr int kWarpLoad = 4, kWarpMma = 5;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&sm.kv_full[s], 1);
      mbar_init(&sm.kv_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], kCompute);
      mbar_init(&sm.pv_done[i], 1);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.o_empty[i], kCompute);
    }
    for (int i = 0; i < kItemRing; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], 1 + 4);  // the issuing thread, four compute warps
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
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  // Q rows the boxes do not fill (N past the unit's heads) stay zero: their
  // columns of S are never used, and cost nothing as zeros.
  for (int i = tid; i < (int)sizeof(sm.q) / 16; i += kDecodeThreads)
    reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  wait_prior_grid();
  PagedWalk walk;
  paged_plan(p, ph, sm.scan, walk);

  auto take_item = [&](int m, bool& ok) -> PagedItem {
    const int slot = m % kItemRing;
    PagedItem it;
    it.end = 1;
    if (ok) ok = mbar_wait(&sm.item_full[slot], (m / kItemRing) & 1, p.status, abortf, kSitePgItemFull);
    if (ok) it = sm.item[slot];
    return it;
  };

  if (warp == kWarpLoad) {
    // ------------------------------------------------------------ producer
    const int lane = (int)lane_id();
    int c = 0, n_q = 0;
    bool ok = true;
    if (walk.g >= walk.hi && lane == 0) {
      PagedRec r = {};
      r.total = walk.total;
      *reinterpret_cast<PagedRec*>(ph.rec + blockIdx.x * kPagedRecBytes) = r;
    }
    for (int m = 0; ok; ++m) {
      const int is = m % kItemRing;
      if (m >= kItemRing)
        ok = mbar_wait(&sm.item_empty[is], (m / kItemRing - 1) & 1, p.status, abortf, kSitePgItemEmpty);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const PagedItem it = paged_next(p, ph, walk);
      if (lane == 0) {
        sm.item[is] = it;
        mbar_arrive(&sm.item_full[is]);
      }
      if (it.end) break;
      if (it.nj == 0) continue;
      PagedPages pages;
      paged_pages_begin(p, ph, it, pages);
      const int qb = n_q & 1;
      if (n_q >= 2)
        ok = mbar_wait(&sm.q_empty[qb], ((n_q >> 1) - 1) & 1, p.status, abortf, kSitePgQEmpty);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sm.q_full[qb], ph.tile_tokens * p.G * D * 2);
        for (int h = 0; h < D / 64; ++h)
          tma_load_3d(sm.q[qb] + h * (N * 128), &tq, &sm.q_full[qb], h * 64, it.h * p.G, it.tok0);
      }
      ++n_q;
      for (int j = 0; j < it.nj && ok; ++j) {
        for (int w = 0; w < 2; ++w) {
          const int slot = c % S, use = c / S;
          if (use > 0)
            ok = mbar_wait(&sm.kv_empty[slot], (use - 1) & 1, p.status, abortf, kSitePgKvEmpty);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          paged_load_tile<D>(p, w == 0 ? &tk : &tv, pages, it.h, it.key + j * kTile, sm.kv[slot],
                             &sm.kv_full[slot]);
          ++c;
        }
      }
    }
    if (!ok && lane == 0) {
      // Let the copies already issued land before the CTA exits.
      for (int i = n_q - 1; i >= 0 && i >= n_q - 2; --i) drain_wait(&sm.q_full[i & 1], (i >> 1) & 1);
      for (int cc = c - 1; cc >= 0 && cc >= c - S; --cc)
        drain_wait(&sm.kv_full[cc % S], (cc / S) & 1);
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ products
    if (lane_id() == 0) {
      const uint32_t id_s = idesc_bf16(128, N, false, false);
      const uint32_t id_o = idesc_bf16(128, N, true, false);
      bool ok = true;
      int m = 0;                 // items read
      int gs = 0, gp = 0;        // S and P V products issued, over all units
      bool have = false, end = false;  // a unit whose S products are not all issued
      int s_nj = 0, s_j = 0, s_n = -1; // that unit: tiles, tiles issued, its number
      int p_nj = 0, p_j = 0, p_n = 0;  // the unit of the next P V product
      // The next unit with keys, waiting for its record or only if it is there.
      auto fetch = [&](bool wait) {
        while (ok && !have && !end) {
          const int slot = m % kItemRing;
          if (!wait && !mbar_try_wait(smem_u32(&sm.item_full[slot]), (m / kItemRing) & 1)) return;
          const PagedItem it = take_item(m, ok);
          if (!ok) return;
          mbar_arrive(&sm.item_empty[slot]);
          ++m;
          if (it.end) {
            end = true;
          } else if (it.nj > 0) {
            have = true;
            s_nj = it.nj;
            s_j = 0;
            ++s_n;
          }
        }
      };
      auto issue_s = [&] {
        const int qb = s_n & 1;
        if (s_j == 0)
          ok = mbar_wait(&sm.q_full[qb], (s_n >> 1) & 1, p.status, abortf, kSitePgQFull);
        const int c = 2 * gs, slot = c % S;
        if (ok) ok = mbar_wait(&sm.kv_full[slot], (c / S) & 1, p.status, abortf, kSitePgKvFull);
        if (!ok) return;
        tc_fence_after();
        const uint64_t kd = desc_here(sdesc_sw128(smem_u32(sm.kv[slot]), 16, 1024));
        const uint64_t qd = desc_here(sdesc_sw128(smem_u32(sm.q[qb]), 16, 1024));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + Cfg::col_s(gs & 1), desc_plus(kd, (kk >> 2) * (kTile * 128) + (kk & 3) * 32),
                 desc_plus(qd, (kk >> 2) * (N * 128) + (kk & 3) * 32), id_s, kk > 0);
        tc_commit(&sm.s_full[gs & 1]);
        tc_commit(&sm.kv_empty[slot]);
        ++gs;
        if (++s_j == s_nj) {
          tc_commit(&sm.q_empty[qb]);
          have = false;
        }
      };
      auto issue_pv = [&] {
        const int ob = p_n & 1, pb = gp & 1;
        const int c = 2 * gp + 1, slot = c % S;
        ok = mbar_wait(&sm.p_full[pb], (gp >> 1) & 1, p.status, abortf, kSitePgPFull);
        if (ok) ok = mbar_wait(&sm.kv_full[slot], (c / S) & 1, p.status, abortf, kSitePgKvFull);
        if (ok && p_j == 0 && p_n >= 2)
          ok = mbar_wait(&sm.o_empty[ob], ((p_n >> 1) - 1) & 1, p.status, abortf, kSitePgOEmpty);
        if (!ok) return;
        tc_fence_after();
        // V^T: the tile's 64-channel blocks along M.  At d = 64 there is one
        // block; the product's upper 64 rows repeat the tile 8 keys on and
        // are never read.
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
        if (++p_j == p_nj) tc_commit(&sm.o_full[ob]);
      };
      // S runs one tile ahead of P V, into the next unit where it is known.
      int q_nj[2] = {0, 0};  // tiles of the units by parity of their number
      while (ok) {
        if (gs == gp) fetch(true);
        if (!ok) break;
        if (gs == gp) {
          if (!have) break;  // the list's end
          q_nj[s_n & 1] = s_nj;
          issue_s();
          if (!ok) break;
        }
        if (gs == gp + 1) {
          if (!have) fetch(false);
          if (ok && have) {
            q_nj[s_n & 1] = s_nj;
            issue_s();
          }
        }
        if (!ok) break;
        if (p_j == p_nj) {  // the next unit's first product (its S is issued)
          if (gp > 0) ++p_n;
          p_nj = q_nj[p_n & 1];
          p_j = 0;
        }
        issue_pv();
      }
      // Every product issued so far must finish before TMEM is released.
      tc_commit(&sm.drain);
      drain_wait(&sm.drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ compute
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const int lane = tid & 31;
    const float ninf = __int_as_float(0xff800000);
    const float c2 = p.scale_log2;
    // This thread's place in a row of P: its key's 16-byte chunk (swizzled
    // with the row) and byte in it.
    uint8_t* const pt0 = sm.pt[0] + (tid >> 6) * (N * 128) + (tid & 7) * 2;
    const int pchunk = (tid & 63) >> 3;
    bool fail = false;
    int g = 0, n_item = 0;
    for (int m = 0;; ++m) {
      bool ok = !fail;
      const PagedItem it = take_item(m, ok);
      fail = !ok;
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&sm.item_empty[m % kItemRing]);
      const int rows = it.end ? 0 : it.ntok * p.G;
      if (!bound_ok(it.end || (it.tok0 >= 0 && it.tok0 + it.ntok <= p.T && rows <= N && it.h < p.Hkv),
                    p.status, abortf, kChkPgItem))
        fail = true;
      // Keys of the unit's rows: row n is query head n % G of token n / G.
      if (!fail && !it.end && tid < N) {
        int lim = 0;
        if (tid < rows) {
          const int tok = tid / p.G;
          if (ph.whole_batch)
            lim = paged_prefix_limit(p, it.tok0 + tok);
          else
            lim = p.causal ? max(0, min(it.pos0 + tok + 1, it.len)) : it.len;
        }
        sm.lim[tid] = lim;  // 0 for the columns past the unit's rows
      }
      if (compute_any(fail)) break;
      if (it.end) break;
      int min_lim = 0x7fffffff;
      for (int n = 0; n < rows; ++n) min_lim = min(min_lim, sm.lim[n]);
      float mref[N], l[N];
#pragma unroll
      for (int n = 0; n < N; ++n) mref[n] = ninf, l[n] = 0.f;
      const uint32_t colO = tmem + lane_base + Cfg::col_o(n_item & 1);
      bool stop = false;
      for (int j = 0; j < it.nj; ++j, ++g) {
        const int key = it.key + j * kTile + tid;
        const int b = g & 1;
        if (!fail)
          fail = !mbar_wait(&sm.s_full[b], (g >> 1) & 1, p.status, abortf, kSitePgSFull);
        fail = __any_sync(0xffffffffu, fail);  // keep the warp's TMEM accesses converged
        float t[N];
        if (!fail) {
          tc_fence_after();
          load_cols<N>(tmem + lane_base + Cfg::col_s(b), t);
          tc_fence_before();
        } else {
#pragma unroll
          for (int n = 0; n < N; ++n) t[n] = ninf;
        }
#pragma unroll
        for (int n = 0; n < N; ++n) t[n] *= c2;
        if (it.key + (j + 1) * kTile > min_lim) {
#pragma unroll
          for (int n = 0; n < N; ++n)
            if (key >= sm.lim[n]) t[n] = ninf;
        }
        bool grow = false;
#pragma unroll
        for (int n = 0; n < N; ++n) grow |= t[n] > mref[n] + kRescaleSlack;
        if (compute_any(grow || fail)) {
          // Some score outgrew the reference: move every row's to its maximum.
#pragma unroll
          for (int n = 0; n < N; ++n) {
            float x = t[n];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            if (lane == 0) sm.top[warp][n] = x;
          }
          if (compute_any(fail)) {
            stop = true;
            break;
          }
          float alpha[N];
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const float top = fmaxf(fmaxf(fmaxf(sm.top[0][n], sm.top[1][n]),
                                          fmaxf(sm.top[2][n], sm.top[3][n])),
                                    mref[n]);
            alpha[n] = top == ninf ? 1.f : ex2_approx(mref[n] - top);
            mref[n] = top;
            l[n] *= alpha[n];
          }
          if (j > 0) {
            // O holds the unit's earlier tiles once their products are done.
            if (!mbar_wait(&sm.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, p.status, abortf,
                           kSitePgPvDone))
              fail = true;
            fail = __any_sync(0xffffffffu, fail);
            if (!fail) {
              tc_fence_after();
              float o[N];
              load_cols<N>(colO, o);
#pragma unroll
              for (int n = 0; n < N; ++n) o[n] *= alpha[n];
              store_cols<N>(colO, o);
              tc_fence_before();
            }
          }
        }
        // P's buffer is free once the product before last has read it.
        if (!fail && g >= 2)
          fail = !mbar_wait(&sm.pv_done[b], ((g >> 1) - 1) & 1, p.status, abortf, kSitePgPvDone);
        if (!fail) {
          uint8_t* const pt = pt0 + b * (N * kTile * 2);
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const float x = ex2_approx(t[n] - (mref[n] == ninf ? 0.f : mref[n]));
            l[n] += x;
            *reinterpret_cast<__nv_bfloat16*>(pt + n * 128 + ((pchunk ^ (n & 7)) << 4)) =
                __float2bfloat16(x);
          }
          if (it.key + (j + 1) * kTile > it.k_hi && key >= it.k_hi) {
            // Slots past the unit's keys may hold anything, and 0 * NaN is
            // NaN: their value rows become zero.
            const int c = 2 * g + 1, slot = c % S;
            fail = !mbar_wait(&sm.kv_full[slot], (c / S) & 1, p.status, abortf, kSitePgKvFull);
            if (!fail) {
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                for (int i = 0; i < 8; ++i)
                  *reinterpret_cast<uint4*>(sm.kv[slot] + h * (kTile * 128) + tid * 128 + i * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&sm.p_full[b]);
        }
      }
      if (stop) break;
      // ------------------------------------------------------ the unit's result
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float x = l[n];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) sm.sum[warp][n] = x;
        if (tid == n) sm.lse2[n] = mref[n];
      }
      if (compute_any(fail)) break;
      const bool merge = it.first && ph.pre_o != nullptr;
      if (tid < N) {
        const float sum = (sm.sum[0][tid] + sm.sum[1][tid]) + (sm.sum[2][tid] + sm.sum[3][tid]);
        float lse2 = sum > 0.f ? sm.lse2[tid] + __log2f(sum) : (sum == 0.f ? ninf : sum);
        float own = sum == 0.f ? 0.f : 1.f / sum, pre = 0.f;
        if (tid < rows) {
          const int tok = it.tok0 + tid / p.G, head = it.h * p.G + tid % p.G;
          const long long row = (long long)tok * p.Hq + head;
          if (merge) {
            const float other = ph.pre_lse[row], top = fmaxf(lse2, other);
            if (top != ninf) {
              const float wa = exp2f(lse2 - top), wb = exp2f(other - top), s = wa + wb;
              own *= wa / s;
              pre = wb / s;
              lse2 = top + log2f(s);
            }
          }
          if (it.slot >= 0)
            ph.slot_lse[((long long)blockIdx.x * 2 + it.slot) * ph.slot_rows + tid] = lse2;
          else if (ph.out_lse)
            ph.out_lse[row] = lse2;
          else
            p.lse[row] = lse2 == ninf ? ninf : lse2 * kLn2;
        }
        sm.f_own[tid] = own;
        sm.f_pre[tid] = pre;
      }
      if (it.nj > 0)
        fail = !mbar_wait(&sm.o_full[n_item & 1], (n_item >> 1) & 1, p.status, abortf, kSitePgOFull);
      fail = compute_any(fail);
      if (fail) break;
      float o[N];
      if (it.nj > 0) {
        tc_fence_after();
        load_cols<N>(colO, o);
        tc_fence_before();
        mbar_arrive(&sm.o_empty[n_item & 1]);
        ++n_item;
      } else {
#pragma unroll
        for (int n = 0; n < N; ++n) o[n] = 0.f;
      }
      if (tid < D) {
        int tok = it.tok0, gh = 0;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          if (n < rows) {
            const long long at = ((long long)tok * p.Hq + it.h * p.G + gh) * D + tid;
            const float w = sm.f_own[n];
            float x = w == 0.f ? 0.f : o[n] * w;
            if (merge) {
              const float wp = sm.f_pre[n];
              if (wp != 0.f) x += wp * ph.pre_o[at];
            }
            if (it.slot >= 0)
              ph.slot_o[(((long long)blockIdx.x * 2 + it.slot) * ph.slot_rows + n) * D + tid] = x;
            else if (ph.out_o)
              ph.out_o[at] = x;
            else
              p.o[at] = __float2bfloat16(x);
          }
          if (++gh == p.G) gh = 0, ++tok;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

// Joins the parts of the units that were shared between CTAs.  A block looks
// at one boundary between CTAs and kRows rows of the unit across it; it has
// work if the boundary is the first inside its unit.  kWarps warps share a
// row's parts (few rows and many parts when decoding, the reverse for
// prompts); the parts are added in list order within a warp and the warps'
// sums in order, so the result does not depend on timing.
template <int D, int kWarps>
__global__ void __launch_bounds__(256) fa_paged_merge_kernel(const PagedParams p,
                                                             const PagedPhase ph) {
  wait_prior_grid();
  constexpr int kPer = D / 32, kRows = 8 / kWarps;
  __shared__ float part_o[8][D], part_l[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedRec rec = *reinterpret_cast<const PagedRec*>(ph.rec + blockIdx.x * kPagedRecBytes);
  if (!rec.split) return;
  const long long active = paged_active(rec.total, p.ctas);
  const long long before = paged_lo(rec.total, active, (long long)blockIdx.x - 1);
  if (before > rec.unit_start) return;  // an earlier boundary has the unit
  const int row = blockIdx.y * kRows + warp / kWarps;
  // Row of the unit -> token and head: Q tiles of tile_tokens tokens, 128 (or
  // slot_rows) rows apart.
  const int in_tile = row % kTile;
  const int tok = (row / kTile) * ph.tile_tokens + in_tile / p.G;
  const bool valid = in_tile < ph.tile_tokens * p.G && tok < rec.ntok;
  if (kRows == 1 && !valid) return;
  const float ninf = __int_as_float(0xff800000);
  const int c0 = (int)blockIdx.x - 1;  // the unit's first CTA, in its last segment's slot
  const int c1 = (int)paged_owner(rec.total, active, rec.unit_end - 1);
  const int n = c1 - c0 + 1;
  auto slot_of = [&](int i) -> long long {
    const int slot = i == 0 && before < rec.unit_start ? 1 : 0;
    return ((long long)(c0 + i) * 2 + slot) * ph.slot_rows + row;
  };
  float m = ninf;
  if (valid)
    for (int i = lane; i < n; i += 32) m = fmaxf(m, ph.slot_lse[slot_of(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float acc[kPer], sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  if (valid && m != ninf) {
    constexpr int kBatch = 4;
    for (int i0 = warp % kWarps; i0 < n; i0 += kBatch * kWarps) {
      float v[kBatch][kPer], w[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * kWarps;
        w[b] = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[b][e] = 0.f;
        if (i < n) {
          const long long s = slot_of(i);
          w[b] = ph.slot_lse[s];
          const float* src = ph.slot_o + s * D + lane * kPer;
          if constexpr (kPer == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[b][0] = x.x, v[b][1] = x.y, v[b][kPer - 2] = x.z, v[b][kPer - 1] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[b][0] = x.x, v[b][1] = x.y;
          }
        } else {
          w[b] = ninf;
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float e = exp2f(w[b] - m);
        sum += e;
        if (e != 0.f) {
#pragma unroll
          for (int x = 0; x < kPer; ++x) acc[x] += e * v[b][x];
        }
      }
    }
  }
  if constexpr (kWarps > 1) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) part_o[warp][lane * kPer + e] = acc[e];
    if (lane == 0) part_l[warp] = sum;
    __syncthreads();
    if (warp % kWarps != 0) return;
    for (int w = 1; w < kWarps; ++w) {
      sum += part_l[warp + w];
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] += part_o[warp + w][lane * kPer + e];
    }
  }
  if (!valid) return;
  const float inv = m == ninf ? 0.f : 1.f / sum;
  const long long out = (long long)(rec.tok0 + tok) * p.Hq + rec.h * p.G + in_tile % p.G;
  const float lse2 = m == ninf ? ninf : m + log2f(sum);
  int no_abort = 0;
  if (!bound_ok(rec.tok0 + tok < p.T && rec.h < p.Hkv, p.status, &no_abort, kChkPgRow)) return;
  if (ph.out_o) {
    float* dst = ph.out_o + out * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) dst[e] = acc[e] * inv;
    if (lane == 0) ph.out_lse[out] = lse2;
  } else {
    __nv_bfloat16* dst = p.o + out * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0) p.lse[out] = m == ninf ? ninf : lse2 * kLn2;
  }
}

template <int D, int N>
int launch_decode(const PagedMaps& t, const PagedParams& p, const PagedPhase& ph,
                  const cudaLaunchConfig_t& base) {
  static_assert(sizeof(DecodeSmem<D, N>) + 1024 <= 232448,
                "decode shared memory above the 227 KB a CTA may have");
  cudaLaunchConfig_t c = base;
  c.blockDim = dim3(kDecodeThreads, 1, 1);
  c.dynamicSmemBytes = sizeof(DecodeSmem<D, N>) + 1024;
  if (cudaFuncSetAttribute(fa_paged_decode_kernel<D, N>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)c.dynamicSmemBytes) != cudaSuccess ||
      cudaLaunchKernelEx(&c, fa_paged_decode_kernel<D, N>, t.q, t.k, t.v, p, ph) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

template <int D>
int launch_merge(const PagedParams& p, const PagedPhase& ph, const cudaLaunchConfig_t& base) {
  cudaLaunchConfig_t c = base;
  c.blockDim = dim3(256, 1, 1);
  c.dynamicSmemBytes = 0;
  cudaError_t e;
  if (ph.slot_rows <= kPagedDecodeRows) {
    c.gridDim = dim3((unsigned)p.ctas, (unsigned)ph.slot_rows, 1);
    e = cudaLaunchKernelEx(&c, fa_paged_merge_kernel<D, 8>, p, ph);
  } else {
    c.gridDim = dim3((unsigned)p.ctas, (unsigned)ph.slot_rows / 8, 1);
    e = cudaLaunchKernelEx(&c, fa_paged_merge_kernel<D, 1>, p, ph);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

// One phase: its attention kernel, then the merge of its split units.
template <int D>
int launch_phase(const PagedParams& p, PagedPhase ph, int rows, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)p.ctas, 1, 1);
  c.stream = stream;
  c.attrs = pdl;
  c.numAttrs = 1;
  const int tile_rows = rows <= kPagedDecodeRows ? rows : kTile;
  ph.tile_tokens = tile_rows / p.G;
  ph.unit_tokens = rows <= kPagedDecodeRows ? ph.tile_tokens : 2 * ph.tile_tokens;
  ph.slot_rows = rows;
  PagedMaps t;
  int rc;
  if ((rc = make_tmap_rows(p.q, p.Hq, p.T, p.q_stride, D, p.G, ph.tile_tokens, &t.q)) != FA_OK ||
      (rc = make_tmap_bhnd_rows(p.k_pages, p.num_pages * p.Hkv, p.page_size, D,
                                p.page_size < kTile ? p.page_size : kTile, &t.k)) != FA_OK ||
      (rc = make_tmap_bhnd_rows(p.v_pages, p.num_pages * p.Hkv, p.page_size, D,
                                p.page_size < kTile ? p.page_size : kTile, &t.v)) != FA_OK)
    return rc;
  switch (rows) {
    case 16: rc = launch_decode<D, 16>(t, p, ph, c); break;
    case 32: rc = launch_decode<D, 32>(t, p, ph, c); break;
    case 64: rc = launch_decode<D, 64>(t, p, ph, c); break;
    default: rc = launch_paged_prompt(t, p, ph, D, c); break;
  }
  if (rc != FA_OK) return rc;
  return launch_merge<D>(p, ph, c);
}

template <int D>
int launch_paged_d(const PagedParams& p, cudaStream_t stream) {
  const PagedForm f = paged_form(p.T, p.G, p.max_q, p.prefix_len);
  const PagedWorkspace w = paged_workspace_layout(p.T, p.Hq, D, f);
  PagedPhase ph = {};
  ph.rec = p.workspace + w.rec;
  ph.slot_o = reinterpret_cast<float*>(p.workspace + w.slot_o);
  ph.slot_lse = reinterpret_cast<float*>(p.workspace + w.slot_lse);
  if (f.share) {
    PagedPhase pre = ph;
    pre.whole_batch = 1;
    pre.out_o = reinterpret_cast<float*>(p.workspace + w.pre_o);
    pre.out_lse = reinterpret_cast<float*>(p.workspace + w.pre_lse);
    const int rc = launch_phase<D>(p, pre, f.prefix_rows, stream);
    if (rc != FA_OK) return rc;
    ph.key0 = p.prefix_len;
    ph.pre_o = pre.out_o;
    ph.pre_lse = pre.out_lse;
  }
  return launch_phase<D>(p, ph, f.rows, stream);
}

}  // namespace

int launch_fwd_paged(const PagedParams& p, int d, cudaStream_t stream) {
  return d == 128 ? launch_paged_d<128>(p, stream) : launch_paged_d<64>(p, stream);
}

}  // namespace fa
