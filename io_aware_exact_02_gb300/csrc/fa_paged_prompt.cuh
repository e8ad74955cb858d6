// fa_paged_prompt.cuh -- attention over a paged key/value cache for many query
// rows to a key/value head: prompt chunks, mixed batches, and a shared prefix
// attended by the rows of a whole batch.  The list of units and its split over
// the CTAs are described in fa_paged.cuh.
//
// Bound by the tensor core.  A unit is two Q tiles of up to 128 rows of one
// key/value head, a row being one of the G query heads of a token (128 / G
// tokens to a tile); both tiles share each K and V tile.  Two softmax
// warpgroups, one per Q tile and one thread per row, take turns with the
// tensor core: while one exponentiates, the other tile's products run.  The
// softmax step is the dense forward's (fa_softmax.cuh).
//
// Warps: 0-3 and 4-7 softmax (and results) of Q tiles 0 and 1, 8 and 10 load K
// and V (TMA: a lane per page box), 9 issues the products, 11 is idle.  Tensor
// memory: S / P of the tiles at columns 0 and 128, O at 256 and 256 + d.
//
// 4 x 1,024 rows over up to 4K keys (32 query, 8 key/value heads, d = 128, the
// merge included): 173 us, 1,390 TFLOP/s.  A step of both Q tiles takes 2,700
// cycles against 2,600 of its products at the library's rate, the end of a
// unit 5,400 (700 for the last product, 3,000 for O, then the next unit's
// record and scores).
#pragma once

#include <type_traits>

#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_paged.cuh"
#include "fa_paged4_tiles.cuh"
#include "fa_softmax.cuh"
#include "sm100_ptx.cuh"

namespace fa {

constexpr int kPromptRing = 4;

template <int D>
struct PromptCfg {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr uint32_t kTmemCols = 512;
  static __device__ __forceinline__ uint32_t col_s(int t) { return (uint32_t)t * 128u; }
  static __device__ __forceinline__ uint32_t col_o(int t) { return 256u + (uint32_t)t * D; }
};

template <int D>
struct alignas(1024) PromptSmem {
  uint8_t q[2][PromptCfg<D>::kTileBytes];
  uint8_t kv[PromptCfg<D>::kStages][PromptCfg<D>::kTileBytes];
  uint8_t out[8][4096];  // a softmax warp's 32 rows x 128 bytes on their way out
  uint64_t q_full, q_empty, q_half;
  uint64_t kv_full[PromptCfg<D>::kStages], kv_empty[PromptCfg<D>::kStages];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_empty[2];
  uint64_t item_full[kPromptRing], item_empty[kPromptRing];
  uint64_t drain;
  PagedItem item[kPromptRing];
  PagedScan scan;
  uint32_t tmem_base;
  int abort_flag;
};

// Key tiles of the segment that Q tile t's rows see (0: it has no rows, or
// they see none).
__device__ __forceinline__ int tile_steps(const PagedParams& p, const PagedPhase& ph,
                                          const PagedItem& it, int t) {
  if (t * ph.tile_tokens >= it.ntok) return 0;
  int hi = it.len;
  if (p.causal && !ph.whole_batch)
    hi = min(it.pos0 + min((t + 1) * ph.tile_tokens, it.ntok), it.len);
  const int x = hi - it.key;
  return x <= 0 ? 0 : min((x + kTile - 1) / kTile, it.nj);
}

// A softmax warp's rows of O out of tensor memory (at colO; ~0: zeros), times
// `own`, plus `pre` times row `row` of pre_o (if given), to row dst_row (none
// if negative) of `wide` (fp32) or of o (bf16); slot: the warp's first row where
// wide is a slot.  A thread has a row, but rows
// are stored by lanes that share them: 128 bytes of the warp's 32 rows at a
// time through `out`, 16-byte chunk c of row r at c ^ (r % 8).  (A thread
// storing its own row wrote 16 of its 256 or 512 bytes at a time: 10,000
// cycles a unit.)  Not inlined: the softmax loop around it needs every
// register, and addresses computed here would be kept through it.
template <int D>
__device__ __noinline__ void store_rows(uint32_t colO, float own, float pre, long long row,
                                        long long dst_row, uint8_t* out, float* wide, float* slot,
                                        const float* pre_o, __nv_bfloat16* o) {
  const int lane = (int)lane_id(), e = lane & 7;
  uint8_t* const mine = out + lane * 128;
  if (slot != nullptr && pre_o == nullptr) {
    // The warp's 32 rows of a slot lie one after another, and rows that are
    // none may be written too.
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = 0u;
      if (colO != ~0u) {
        tmem_ld32(colO + c * 32, w);
        tmem_wait_ld(w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = own == 0.f ? 0.f : __uint_as_float(w[4 * i + k]) * own;
        *reinterpret_cast<float4*>(mine + ((i ^ (lane & 7)) << 4)) =
            make_float4(x[0], x[1], x[2], x[3]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = i * 4 + lane / 8;
        *reinterpret_cast<float4*>(slot + rr * D + c * 32 + e * 4) =
            *reinterpret_cast<const float4*>(out + rr * 128 + ((e ^ (rr & 7)) << 4));
      }
      __syncwarp();
    }
    return;
  }
  if (wide != nullptr || pre_o != nullptr) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = 0u;
      if (colO != ~0u) {
        tmem_ld32(colO + c * 32, w);
        tmem_wait_ld(w);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i)
        w[i] = own == 0.f ? 0u : __float_as_uint(__uint_as_float(w[i]) * own);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(mine + ((i ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      __syncwarp();
#pragma unroll 2
      for (int i = 0; i < 8; ++i) {
        const int rr = i * 4 + lane / 8;
        const long long to = __shfl_sync(0xffffffffu, dst_row, rr);
        const long long from = __shfl_sync(0xffffffffu, row, rr);
        const float f = __shfl_sync(0xffffffffu, pre, rr);
        if (to < 0) continue;
        float4 x = *reinterpret_cast<const float4*>(out + rr * 128 + ((e ^ (rr & 7)) << 4));
        const int col = c * 32 + e * 4;
        if (f != 0.f) {
          const float4 y = *reinterpret_cast<const float4*>(pre_o + from * D + col);
          x.x += f * y.x, x.y += f * y.y, x.z += f * y.z, x.w += f * y.w;
        }
        if (wide != nullptr)
          *reinterpret_cast<float4*>(wide + to * D + col) = x;
        else
          *reinterpret_cast<uint2*>(o + to * D + col) =
              make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
      }
      __syncwarp();
    }
    return;
  }
#pragma unroll 1
  for (int c = 0; c < D / 64; ++c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = 0u;
      if (colO != ~0u) {
        tmem_ld32(colO + c * 64 + h * 32, w);
        tmem_wait_ld(w);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = own == 0.f ? 0u
                          : pack_bf16x2(__uint_as_float(w[2 * i]) * own,
                                        __uint_as_float(w[2 * i + 1]) * own);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(mine + (((4 * h + i) ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int rr = i * 4 + lane / 8;
      const long long to = __shfl_sync(0xffffffffu, dst_row, rr);
      if (to >= 0)
        *reinterpret_cast<uint4*>(o + to * D + c * 64 + e * 8) =
            *reinterpret_cast<const uint4*>(out + rr * 128 + ((e ^ (rr & 7)) << 4));
    }
    __syncwarp();
  }
}

// The same for 32 rows of o that are all valid and whole tokens: a box of 64
// channels at a time, stored by TMA (row r's 16-byte chunk c at c ^ (r % 8), as
// its swizzle wants it): 3,000 cycles a unit against 5,700 of store_rows.
template <int D>
__device__ __noinline__ void store_box(uint32_t colO, float own, uint8_t* out,
                                       const CUtensorMap* to, int head, int tok) {
  const int lane = (int)lane_id();
  uint8_t* const mine = out + lane * 128;
#pragma unroll 1
  for (int c = 0; c < D / 64; ++c) {
    uint32_t w[2][16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t x[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = 0u;
      if (colO != ~0u) {
        tmem_ld32(colO + c * 64 + h * 32, x);
        tmem_wait_ld(x);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[h][i] = own == 0.f ? 0u
                             : pack_bf16x2(__uint_as_float(x[2 * i]) * own,
                                           __uint_as_float(x[2 * i + 1]) * own);
    }
    if (c > 0) {
      if (lane == 0) bulk_wait_group_read0();
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint4*>(mine + ((i ^ (lane & 7)) << 4)) =
          make_uint4(w[i / 4][4 * (i % 4)], w[i / 4][4 * (i % 4) + 1], w[i / 4][4 * (i % 4) + 2],
                     w[i / 4][4 * (i % 4) + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(to, out, c * 64, head, tok);
      bulk_commit_group();
    }
  }
}

// The prompt kernel's work on CTA `cta` of the `ctas` that share the phase's
// list.  kStarted: the caller has waited for the prior grid.
//
// kFour: over the cache in 4 bits (fa_kv4.cuh).  Four more warps, 12-15, turn its
// codes into fp16 tiles, warp 8 has the list and Q only, 10 is idle too; the
// products run in fp16, and the softmax warps scale each row of Q to its range
// first.  kWhole: the tiles are in fp16 already, and warp 10 loads them.
template <int D, bool kNeg, bool kStarted, bool kFour = false, bool kWhole = false>
__device__ __forceinline__ void prompt_cta(
    const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv, const CUtensorMap* to,
    const std::conditional_t<kFour, Paged4Params, PagedParams>& p, const PagedPhase& ph, int cta,
    int ctas, uint8_t* smem_raw) {
  using Cfg = PromptCfg<D>;
  constexpr int S = Cfg::kStages;
  PromptSmem<D>& sm = *reinterpret_cast<PromptSmem<D>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abortf = &sm.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5;
  constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpLoadV = 10, kWarpTiles = 12;
  constexpr bool kMakes = kFour && !kWhole;  // (has warps that make tiles)
  constexpr int kThreads = kMakes ? kPaged4Threads : kPagedThreads;
  constexpr int kRegsCompute = kMakes ? kPaged4RegsCompute : kPagedRegsCompute;
  constexpr int kRegsLoad = kMakes ? kPaged4RegsList : kPagedRegsLoad;

  if (tid == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    if constexpr (kFour) mbar_init(&sm.q_half, 256);
    for (int s = 0; s < S; ++s) {
      mbar_init(&sm.kv_full[s], kMakes ? 4 : 1);
      mbar_init(&sm.kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_half[t], 128);
      mbar_init(&sm.p_full[t], 128);
      mbar_init(&sm.o_full[t], 1);
      mbar_init(&sm.o_empty[t], 128);
    }
    for (int i = 0; i < kPromptRing; ++i) {
      mbar_init(&sm.item_full[i], 1);
      // Read by the issuing thread, the V warp (kMakes: the four that make tiles)
      // and the eight softmax warps.
      mbar_init(&sm.item_empty[i], (kMakes ? 5 : 2) + 8);
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
    if constexpr (!kFour) {
      prefetch_tmap(tk);
      prefetch_tmap(tv);
    }
  }
  if (ph.tile_tokens * p.G < kTile) {
    // Rows no box fills: any finite values do (their results are not stored),
    // zeros never move the running maximum.
    for (int i = tid; i < (int)sizeof(sm.q) / 16; i += kThreads)
      reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
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

  auto take_item = [&](int m, bool& ok) -> PagedItem {
    const int slot = m % kPromptRing;
    PagedItem it;
    it.end = 1;
    ok = mbar_wait(&sm.item_full[slot], (m / kPromptRing) & 1, p.status, abortf, kSitePgItemFull);
    if (ok) it = sm.item[slot];
    return it;
  };

  if (warp == kWarpLoad) {
    // ------------------------------------------------------------ Q and K
    setmaxnreg_dec<kRegsLoad>();
    int n_q = 0;  // units loaded
    auto load_q = [&](const PagedItem& it) {
      if (n_q > 0 &&
          !mbar_wait(&sm.q_empty, (n_q - 1) & 1, p.status, abortf, kSitePgQEmpty))
        return false;
      if (lane_id() == 0) {
        mbar_arrive_expect_tx(&sm.q_full, 2 * ph.tile_tokens * p.G * D * 2);
        for (int t = 0; t < 2; ++t)
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sm.q[t] + h * 16384, tq, &sm.q_full, h * 64, it.h * p.G,
                        it.tok0 + t * ph.tile_tokens);
      }
      ++n_q;
      return true;
    };
    if constexpr (kFour)
      paged4_produce_items<kPromptRing>(p, ph, sm, walk, cta, ctas, load_q);
    else
      paged_produce_k<D, S, kPromptRing>(p, ph, sm, tk, walk, cta, ctas, 1, load_q);
    if (*abortf && lane_id() == 0 && n_q > 0) drain_wait(&sm.q_full, (n_q - 1) & 1);
    __syncwarp();
  } else if (warp == kWarpLoadV) {
    // ------------------------------------------------------------ V
    setmaxnreg_dec<kRegsLoad>();
    if constexpr (kWhole)
      paged4_load_tiles<D, S, kPromptRing>(p, sm);
    else if constexpr (!kFour)
      paged_produce_v<D, S, kPromptRing>(p, sm, tv, nullptr);
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ products
    setmaxnreg_dec<kRegsLoad>();
    if (lane_id() == 0) {
      // (In the descriptor, fp16 is 0 where bf16 is 1.)
      constexpr uint32_t kTypes = kFour ? 1u << 7 | 1u << 10 : 0u;
      const uint32_t id_s = idesc_bf16(128, 128, false, false) & ~kTypes;
      const uint32_t id_o = idesc_bf16(128, D, false, true) & ~kTypes;
      const uint32_t q_addr[2] = {smem_u32(sm.q[0]), smem_u32(sm.q[1])};
      uint32_t p_par[2] = {0, 0};
      int n_o[2] = {0, 0};  // units whose O_t was begun
      int cb = 0, n_q = 0;
      bool ok = true;
      auto issue_s = [&](int t, int slot) {
        const uint64_t qd = desc_here(sdesc_sw128(q_addr[t], 16, 1024));
        const uint64_t kd = desc_here(sdesc_sw128(smem_u32(sm.kv[slot]), 16, 1024));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_ss(tmem + Cfg::col_s(t), desc_plus(qd, off), desc_plus(kd, off), id_s, kk > 0);
        }
        tc_commit(&sm.s_full[t]);
      };
      // O_t += P_t V; the unit's first product overwrites O_t, once softmax t
      // has read the previous unit's.
      auto issue_pv = [&](int t, int slot, bool accumulate) -> bool {
        if (!mbar_wait(&sm.p_half[t], p_par[t], p.status, abortf, kSitePgPHalf)) return false;
        if (!accumulate) {
          if (n_o[t] > 0 &&
              !mbar_wait(&sm.o_empty[t], (n_o[t] - 1) & 1, p.status, abortf, kSitePgOEmpty))
            return false;
          ++n_o[t];
        }
        tc_fence_after();
        const uint64_t vd = desc_here(sdesc_sw128(smem_u32(sm.kv[slot]), 16384, 1024));
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk) {
          if (kk == kTile / 32) {  // the second half of P
            const bool r = mbar_wait(&sm.p_full[t], p_par[t], p.status, abortf, kSitePgPFull);
            p_par[t] ^= 1;
            if (!r) return false;
            tc_fence_after();
          }
          mma_ts(tmem + Cfg::col_o(t), tmem + Cfg::col_s(t) + kk * 8, desc_plus(vd, kk * 2048),
                 id_o, (accumulate || kk > 0) ? 1u : 0u);
        }
        return true;
      };
      auto wait_full = [&](int c) -> bool {
        return mbar_wait(&sm.kv_full[c % S], (c / S) & 1, p.status, abortf, kSitePgKvFull);
      };
      for (int m = 0; ok; ++m) {
        const PagedItem it = take_item(m, ok);
        if (!ok) break;
        mbar_arrive(&sm.item_empty[m % kPromptRing]);
        if (it.end) break;
        const int n_t[2] = {tile_steps(p, ph, it, 0), tile_steps(p, ph, it, 1)};
        const int nmax = max(n_t[0], n_t[1]);
        if (nmax == 0) continue;
        ok = mbar_wait(kFour ? &sm.q_half : &sm.q_full, n_q & 1, p.status, abortf, kSitePgQFull);
        if (ok) ok = wait_full(cb);
        if (!ok) break;
        ++n_q;
        tc_fence_after();
        for (int t = 0; t < 2; ++t)
          if (n_t[t] > 0) issue_s(t, cb % S);
        tc_commit(&sm.kv_empty[cb % S]);
        if (nmax == 1) tc_commit(&sm.q_empty);
        // Key tile j: P_t(j-1) V, then S_t(j), for each Q tile that has them.
        for (int j = 1; j < nmax && ok; ++j) {
          const int kc = cb + 2 * j, vc = kc - 1;
          ok = wait_full(kc) && wait_full(vc);
          for (int t = 0; t < 2 && ok; ++t) {
            if (j - 1 >= n_t[t]) continue;
            ok = issue_pv(t, vc % S, j > 1);
            if (!ok) break;
            if (j < n_t[t])
              issue_s(t, kc % S);
            else
              tc_commit(&sm.o_full[t]);
          }
          if (!ok) break;
          tc_commit(&sm.kv_empty[vc % S]);
          tc_commit(&sm.kv_empty[kc % S]);
          if (j == nmax - 1) tc_commit(&sm.q_empty);
        }
        if (!ok) break;
        const int vc = cb + 2 * nmax - 1;
        ok = wait_full(vc);
        for (int t = 0; t < 2 && ok; ++t) {
          if (n_t[t] != nmax) continue;
          ok = issue_pv(t, vc % S, nmax > 1);
          if (ok) tc_commit(&sm.o_full[t]);
        }
        if (ok) tc_commit(&sm.kv_empty[vc % S]);
        cb += 2 * nmax;
      }
      // Every product issued so far must finish before TMEM is released.
      tc_commit(&sm.drain);
      drain_wait(&sm.drain, 0);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<kRegsCompute>();
    const int t = warp >> 2;  // Q tile
    const int r = tid & 127;  // row of the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t colS = tmem + lane_base + Cfg::col_s(t);
    const uint32_t colO = tmem + lane_base + Cfg::col_o(t);
    const float ninf = __int_as_float(0xff800000);
    float c2 = p.scale_log2;  // nonzero: a zero scale arrives as a tiny positive one
    [[maybe_unused]] int n_q = 0;
    const int row_tok = t * ph.tile_tokens + r / p.G, row_head = r % p.G;
    uint32_t s_par = 0;
    int n_o = 0;  // units with keys for this tile
    int cb = 0;   // ring uses before the current unit
    bool ok = true;
    for (int m = 0; ok; ++m) {
      const PagedItem it = take_item(m, ok);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      __syncwarp();  // every lane has read the record
      if (lane_id() == 0) mbar_arrive(&sm.item_empty[m % kPromptRing]);
      if (it.end) break;
      const int n_t = tile_steps(p, ph, it, t);
      const int nmax = max(n_t, tile_steps(p, ph, it, 1 - t));
      const bool valid = r < ph.tile_tokens * p.G && row_tok < it.ntok;
      if (!warp_bound_ok(!valid || (it.tok0 >= 0 && it.tok0 + row_tok < p.T && it.h < p.Hkv),
                         p.status, abortf, kChkPgItem)) {
        ok = false;
        break;
      }
      int lim = 0;  // the row sees keys below it
      if (valid) {
        if (ph.whole_batch)
          lim = paged_prefix_limit(p, it.tok0 + row_tok);
        else
          lim = p.causal ? min(it.pos0 + row_tok + 1, it.len) : it.len;
      }
      float m_ref = ninf, l = 0.f;
      if constexpr (kFour) {
        if (nmax > 0) {
          ok = mbar_wait(&sm.q_full, n_q & 1, p.status, abortf, kSitePgQFull);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++n_q;
          c2 = q_row_to_half<D, kNeg>(sm.q[t], r, p.scale_log2 * p.k_scale);
          fence_proxy_async_smem();
          mbar_arrive(&sm.q_half);
        }
      }
      for (int j = 0; j < n_t; ++j) {
        const int key = it.key + j * kTile;
        ok = mbar_wait(&sm.s_full[t], s_par, p.status, abortf, kSitePgSFull);
        if (ok && key + kTile > it.k_hi) {
          // Slots past the unit's keys may hold anything, and 0 * NaN is NaN:
          // their value rows become zero (for each Q tile before its product).
          const int c = cb + 2 * j + 1, slot = c % S;
          ok = mbar_wait(&sm.kv_full[slot], (c / S) & 1, p.status, abortf, kSitePgKvFull);
          if (ok && key + r >= it.k_hi) {
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(sm.kv[slot] + h * 16384 + r * 128 + i * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        ok = __all_sync(0xffffffffu, ok);  // keep the warp's collective TMEM ops converged
        s_par ^= 1;
        if (!ok) break;
        tc_fence_after();
        softmax_tile<D, kNeg, false, kFour>(colS, colO, c2, lim - key, j > 0, m_ref, l,
                                     [&] { mbar_arrive(&sm.p_half[t]); });
        tc_fence_before();
        mbar_arrive(&sm.p_full[t]);
      }
      if (!ok) break;
      cb += 2 * nmax;
      // -------------------------------------------------- the rows' results
      const long long row = (long long)(it.tok0 + row_tok) * p.Hq + it.h * p.G + row_head;
      const bool any = l > 0.f || l != l;
      float lse2 = any ? m_ref + __log2f(l) : ninf;
      float own = any ? 1.f / l : 0.f, pre = 0.f;
      if constexpr (kFour) own *= p.v_scale;
      if (it.first && ph.pre_o != nullptr && valid) {
        const float other = ph.pre_lse[row], top = fmaxf(lse2, other);
        if (top != ninf) {
          const float wa = exp2f(lse2 - top), wb = exp2f(other - top), s = wa + wb;
          own *= wa / s;
          pre = wb / s;
          lse2 = top + log2f(s);
        }
      }
      if (n_t > 0) {
        ok = mbar_wait(&sm.o_full[t], n_o & 1, p.status, abortf, kSitePgOFull);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      const long long slot_row = ((long long)cta * 2 + it.slot) * ph.slot_rows + t * kTile + r;
      if (lane_id() == 0) bulk_wait_group_read0();  // of the last unit's boxes
      __syncwarp();
      // A warp's 32 rows are whole tokens; all of them are the unit's.
      const bool box = ph.box_out && it.slot < 0 && !(it.first && ph.pre_o != nullptr) &&
                       __all_sync(0xffffffffu, valid);
      if (box)
        store_box<D>(n_t > 0 ? colO : ~0u, own, sm.out[warp], to, it.h * p.G,
                     it.tok0 + t * ph.tile_tokens + (warp & 3) * (32 / p.G));
      else
        store_rows<D>(n_t > 0 ? colO : ~0u, own, pre, row,
                      valid ? (it.slot >= 0 ? slot_row : row) : -1, sm.out[warp],
                      it.slot >= 0 ? ph.slot_o : ph.out_o,
                      it.slot >= 0 ? ph.slot_o + (slot_row - lane_id()) * D : nullptr,
                      it.first ? ph.pre_o : nullptr, p.o);
      if (n_t > 0) {
        // O_t may now be overwritten by the next unit's first product.
        tc_fence_before();
        mbar_arrive(&sm.o_empty[t]);
        ++n_o;
      }
      if (valid) {
        if (it.slot >= 0)
          ph.slot_lse[slot_row] = lse2;
        else if (ph.out_lse)
          ph.out_lse[row] = lse2;
        else
          p.lse[row] = lse2 == ninf ? ninf : lse2 * kLn2;
      }
    }
    if (lane_id() == 0) bulk_wait_group0();
    __syncwarp();
  } else if (kMakes && warp >= kWarpTiles) {
    // ------------------------------------------------------------ tiles
    if constexpr (kMakes) {
      setmaxnreg_dec<kPaged4RegsTiles>();
      paged4_produce_tiles<D, S, kPromptRing>(p, sm, warp - kWarpTiles);
    }
  } else {
    // Idle: its registers go to the compute warps.
    setmaxnreg_dec<kRegsLoad>();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

}  // namespace fa
