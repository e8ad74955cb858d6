// fa_paged4_decode.cuh -- attention over a paged cache held in 4 bits for few
// query rows to a key/value head.  The list of units and its split over the CTAs
// are those of fa_paged.cuh, the numbers and their layout those of fa_kv4.cuh.
//
// Keys and values are read once and used by 8 or 16 rows, so the kernel's job is
// to keep memory busy; but 45 bytes a nanosecond and SM are 80 numbers, and each
// has to be turned into a 16-bit operand of the tensor core.  What that costs
// decides the form: an operand in shared memory would be written and read
// there once more (160 and 160 of the 250 bytes a nanosecond that shared memory
// moves), so the products are mma.sync's, whose operands are registers.  Its
// rate (measured: 4.1 ns for a 16 x 8 x 16 product on a quarter of an SM) is a
// third used with 8 rows, two thirds with 16; the conversion of codes (76 pairs
// a nanosecond and SM) is half used.
//
// A warp works alone on blocks of 16 keys of a unit, which arrive in its own ring:
//     S^T [16 keys x rows] = K [16 x d] Q^T,    O^T [d x rows] += V^T [d x 16] P^T
// with keys, then channels, along the 16 rows of the product, so that 8 query
// rows leave none of it unused.  A lane (g, t) = (lane / 4, lane % 4) reads from
// a block channels t d/4 .. of keys g and g + 8, whose order in the first product
// is free, and channels g d/8 .. of the key pairs (2t, 2t + 1) and 8 further on:
// the layout of a block makes each one 16-byte load (d = 64: 8-byte) of
// consecutive addresses.  P goes from the first product's layout to the
// second's by a transposition of 8 x 8 matrices among the warp's registers.
// The reference of a row's exponents is a warp's own, kHalfHeadroom below the first
// step's maximum, and moves only when scores exceed that by kRescaleSlack.  At a unit's end the warps' parts are
// joined through shared memory.
//
// Measured, H_q 32, H_kv 8, d = 128, one row each: 8 sequences of 32K keys 65.9 us (302
// MB: 4.6 TB/s), 64 of up to 4K 46.1, one of 1,000 10.3; 33 of 2K with 1 to 4 rows, 16
// heads, d = 64: 25.1.  The steps alone, by what more keys cost (8 sequences of 128K and
// 256K): 5.9 TB/s, 87% of the copy rate; d = 64 4.7 to 5; with 16 rows, d = 128, 3.5.
// So 14 of the 65.9 us lie around the steps: start, units' ends, and the merge, a
// kernel of 6 to 7 us.  Three CTAs an SM, because
// one's unit end hides behind the others' steps (one CTA of 16 warps: 62.6 us
// instead of 50 for the 64 sequences); steps of two blocks, whose chains of latencies
// hide behind one another (79.6 us instead of 69.2 for the 8).
//
// Warps: 0 .. W-1 load and compute; warp W walks the list and turns each unit's
// query rows into fp16, scaled by a power of two each.  (One warp loading for all
// of them bounded the kernel: 70 ns a block.)
#pragma once

#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_paged.cuh"
#include "fa_softmax.cuh"
#include "sm100_ptx.cuh"

namespace fa {

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16).
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit numbers, two to a lane.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// A vote of `threads` threads on named barrier `id`: true for all when true for
// any.  Also a barrier among them.
__device__ __forceinline__ bool named_vote(int id, int threads, bool x) {
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

// What the end of a unit costs, in 128-key tiles: 2 to 4 us of a CTA, against 1.4
// (d = 64: 0.8) for a tile.
constexpr int kEndTiles = 2;

template <int D, int R>
struct Decode4Cfg {
  static constexpr int kTiles = R / 8;
  static constexpr int kCtas = kPaged4CtasPerSm;  // of an SM
  static constexpr int kWarps = R == 8 ? 4 : 3;  // that compute
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kUnit = 2;  // blocks of a step: the latencies of one hide behind the other's
  static constexpr int kStages = D == 128 ? 2 : 4;  // steps in a warp's ring
  static constexpr int kItems = 4;
};

template <int D, int R>
struct alignas(128) Decode4Smem {
  using Cfg = Decode4Cfg<D, R>;
  static constexpr int W = Cfg::kWarps;
  uint8_t ring[W][Cfg::kStages][Cfg::kUnit * Kv4Block<D>::kBytes];
  float part_o[W][R][D];  // 16-byte chunk c of row r at c ^ (r / 2 % 4)
  uint4 q[2][R / 8 * (D / 32)][32];  // [8 rows, 8 of a lane's channels][lane of the product]
  float part_m[W][R], part_l[W][R];
  float c2[2][R];         // a row's factor from products to exponents
  int lim[2][R];          // the keys that a row sees end here
  uint64_t full[W][Cfg::kStages];
  uint64_t item_full[Cfg::kItems], item_empty[Cfg::kItems];
  uint64_t q_full[2], q_empty[2];
  PagedItem item[Cfg::kItems];
  PagedScan scan;
  int abort_flag;
};

// Keys of a segment.
__device__ __forceinline__ int item_keys(const PagedItem& it) {
  return it.nj == 0 ? 0 : min(it.k_hi - it.key, it.nj * kTile);
}

// The kernel's work on CTA `cta` of `ctas`.  p.Hkv heads of p.G rows each: `subs`
// of them share a key/value head of the cache.
template <int D, int R>
__device__ __forceinline__ void decode4_cta(const Paged4Params& p, const PagedPhase& ph, int subs,
                                            int cta, int ctas, uint8_t* smem_raw) {
  using Cfg = Decode4Cfg<D, R>;
  using Block = Kv4Block<D>;
  constexpr int W = Cfg::kWarps, S = Cfg::kStages, NT = Cfg::kTiles, U = Cfg::kUnit;
  Decode4Smem<D, R>& sm = *reinterpret_cast<Decode4Smem<D, R>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  volatile int* abortf = &sm.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < W * S; i += Cfg::kThreads) mbar_init(&sm.full[0][0] + i, 1);
  if (tid == 0) {
    for (int i = 0; i < Cfg::kItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], W);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], W);
    }
    sm.abort_flag = 0;
  }
  fence_mbar_init();
  __syncthreads();
  launch_dependents();
  wait_prior_grid();
  PagedWalk walk;
  paged_plan<kEndTiles>(p, ph, sm.scan, walk, cta, ctas);

  if (warp == W) {
    // ------------------------------------------------------------ the list, and query rows
    paged_walk_begin<kEndTiles>(p, ph, sm.scan, walk, cta, ctas);
    PagedRec* const rec = reinterpret_cast<PagedRec*>(ph.rec + cta * kPagedRecBytes);
    bool ok = true;
    for (int m = 0; ok; ++m) {
      const PagedItem it = paged_next_weighed<kEndTiles>(p, ph, walk, cta);
      const int is = m % Cfg::kItems, qb = m & 1, rows = it.ntok * p.G;
      if (m >= Cfg::kItems)
        ok = mbar_wait(&sm.item_empty[is], (m / Cfg::kItems - 1) & 1, p.status, abortf,
                       kSitePgItemEmpty);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        sm.item[is] = it;
        mbar_arrive(&sm.item_full[is]);
      }
      if (it.end) {
        if (m == 0 && lane == 0) rec->split = 0;
        break;
      }
      if (!warp_bound_ok(it.tok0 >= 0 && rows <= R && it.tok0 + it.ntok <= p.T && it.h < p.Hkv,
                         p.status, abortf, kChkPgItem))
        break;
      // Lane (g, t) has channels t d/4 .. of row g of each eight, as the product
      // takes them.
      const int g = lane >> 2, t = lane & 3;
      uint4 x[NT][D / 32];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g, tok = r / p.G;
        const __nv_bfloat16* src = p.q + (it.tok0 + tok) * p.q_stride +
                                   (long long)(it.h * p.G + r - tok * p.G) * D + t * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          x[nt][i] = r < rows ? reinterpret_cast<const uint4*>(src)[i] : make_uint4(0u, 0u, 0u, 0u);
      }
      // What the merge needs to know of the CTA's first unit.
      if (m == 0 && lane == 0) {
        *rec = paged4_first_rec(it, walk);
      }
      __syncwarp();
      if (m >= 2) ok = mbar_wait(&sm.q_empty[qb], (m / 2 - 1) & 1, p.status, abortf, kSitePgQEmpty);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g;
        uint32_t w[D / 8];  // pairs of channels
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          w[4 * i] = x[nt][i].x, w[4 * i + 1] = x[nt][i].y, w[4 * i + 2] = x[nt][i].z, w[4 * i + 3] = x[nt][i].w;
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) top = kv4_top(top, w[i]);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = kv4_row_exponent(top);
        const float f = kv4_pow2(e);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          sm.q[qb][nt * (D / 32) + i][lane] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        if (t == 0) {
          sm.c2[qb][r] = r < rows ? p.scale_log2 * p.k_scale * kv4_pow2(-e) : 0.f;
          int lim = 0;
          if (r < rows) lim = p.causal ? max(0, min(it.pos0 + r / p.G + 1, it.len)) : it.len;
          sm.lim[qb][r] = lim;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[qb]);
    }
    return;
  }

  // -------------------------------------------------------------- compute
  const int g = lane >> 2, t = lane & 3;
  const float ninf = __int_as_float(0xff800000);
  bool fail = false;
  int off = 0;  // the warp of the segment's first step: step i is warp (off + i) % W's
  int c = 0;    // steps this warp has had
  int issued = 0;
  // The current segment: this warp's steps, the first one's first key (the next
  // one's is 16 U W further on), where their pages are listed, and the numbers
  // of 32 blocks' pages in the lanes, with the next 32.
  int end = 0, own = 0, key0 = 0, head = 0, rows = 0, tok0 = 0, head0 = 0, oslot = -1, min_lim = 0,
      k_hi = 0, seq = 0, pg = 0, pg2 = 0;
  int ahead = 0, ahead2 = 0;  // the next segment's pages, if it was looked at
  bool looked = false;
  auto key_of = [&](int block) -> int {  // the first key of own block U j + b
    return key0 + 16 * (block / U * (W * U) + block % U);
  };
  auto page_at = [&](int block) -> int {
    const int key = key_of(block);
    return block < own * U && key < k_hi
               ? p.page_table[(long long)seq * p.max_pages + (key >> p.page_shift)]
               : 0;
  };
  // Issues the loads of own step j (c0 steps went before the segment's), a lane
  // to a block.
  auto issue = [&](int j, int c0) {
    const int first = j * U;
    if (j > 0 && (first & 31) == 0) {
      pg = pg2;
      pg2 = page_at(first + 32 + lane);
    }
    const int page = __shfl_sync(0xffffffffu, pg, (first + lane) & 31), slot = (c0 + j) % S;
    const int key = key_of(first + (lane & (U - 1)));
    const bool on = lane < U && key < k_hi, valid = on && page >= 0 && page < p.num_pages;
    const unsigned copies = __ballot_sync(0xffffffffu, valid);
    if (lane == 0) mbar_arrive_expect_tx(&sm.full[warp][slot], __popc(copies) * Block::kBytes);
    if (on && !valid) {  // (the step takes whatever the slot holds)
      int abort_flag = 0;
      report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPage);
    }
    __syncwarp();
    if (valid)
      bulk_load(sm.ring[warp][slot] + lane * Block::kBytes,
                p.pages + kv4_block_at(page, p.Hkv / subs, head, p.page_shift,
                                       key & (p.page_size - 1), Block::kBytes),
                Block::kBytes, &sm.full[warp][slot]);
    __syncwarp();
    ++issued;
  };
  // The warp's part of a segment: how many steps, and the first one's first key.
  auto part = [&](const PagedItem& it, int& first_key) -> int {
    const int n = it.end ? 0 : (item_keys(it) + 16 * U - 1) / (16 * U);
    const int i0 = warp >= off ? warp - off : warp - off + W;
    first_key = it.key + 16 * U * i0;
    return i0 < n ? (n - i0 + W - 1) / W : 0;
  };
  // Asks for the pages of segment m, if it is known by now.
  auto look = [&](int m) {
    const int is = m % Cfg::kItems;
    looked = __all_sync(0xffffffffu, mbar_test_wait(&sm.item_full[is], (m / Cfg::kItems) & 1));
    if (!looked) return;
    const PagedItem& it = sm.item[is];
    int first_key;
    const int steps = part(it, first_key), hi = it.key + item_keys(it);
    const int* const list = p.page_table + (long long)it.b * p.max_pages;
    auto at = [&](int block) -> int {
      const int key = first_key + 16 * (block / U * (W * U) + block % U);
      return block < steps * U && key < hi ? list[key >> p.page_shift] : 0;
    };
    ahead = at(lane);
    ahead2 = at(lane + 32);
  };
  // Takes segment m: its record, its pages, and the first loads.
  auto take = [&](int m) {
    const int is = m % Cfg::kItems;
    if (!fail && !looked)
      fail = !mbar_wait(&sm.item_full[is], (m / Cfg::kItems) & 1, p.status, abortf, kSitePgItemFull);
    fail = __any_sync(0xffffffffu, fail);
    end = own = 0;
    if (fail) return;
    if (!looked) look(m);
    const PagedItem& it = sm.item[is];
    end = it.end;
    own = part(it, key0);
    off = end ? off : (off + (item_keys(it) + 16 * U - 1) / (16 * U)) % W;
    head = it.h / subs;
    rows = it.ntok * p.G;
    tok0 = it.tok0;
    head0 = it.h * p.G;
    oslot = it.slot;
    seq = it.b;
    k_hi = it.key + item_keys(it);
    min_lim = p.causal ? it.pos0 + 1 : it.len;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[is]);
    pg = ahead;
    pg2 = ahead2;
    looked = false;
    for (int j = 0; j < S && j < own; ++j) issue(j, c);
  };
  take(0);
  for (int m = 0;; ++m) {
    const int qb = m & 1;
    float ref[NT][2], l[NT][2], c2[NT][2], o[D / 16][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) ref[nt][e] = 0.f, l[nt][e] = 0.f;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    if (!fail && !end) {
      fail = !mbar_wait(&sm.q_full[qb], (m / 2) & 1, p.status, abortf, kSitePgQFull);
      fail = __any_sync(0xffffffffu, fail);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) c2[nt][e] = sm.c2[qb][nt * 8 + 2 * t + e];
      const int c0 = c;
      for (int j = 0; j < own && !fail; ++j, ++c) {
        const int slot = c % S, key = key0 + 16 * U * W * j;
        fail = !mbar_wait(&sm.full[warp][slot], (c / S) & 1, p.status, abortf, kSitePgKvFull);
        fail = __any_sync(0xffffffffu, fail);
        if (fail) break;
        constexpr int kWords = D / 32;  // of four bytes: a key's, or a value pair's, of this lane
        const uint8_t* const blk = sm.ring[warp][slot];
        // A lane's 16 (d = 64: 8) bytes of the u-th 32 of a block's codes.
        auto words = [&](const uint8_t* codes, int u, uint32_t (&w)[kWords]) {
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(codes + (u * 32 + lane) * 16);
            w[0] = x.x, w[1] = x.y, w[kWords - 2] = x.z, w[kWords - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(codes + (u * 32 + lane) * 8);
            w[0] = x.x, w[1] = x.y;
          }
        };
        uint32_t kw[U][2][kWords], ks[U][2];
#pragma unroll
        for (int b = 0; b < U; ++b)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            words(blk + b * Block::kBytes + Block::k_code(0), u, kw[b][u]);
            const uint8_t* const sc = blk + b * Block::kBytes + Block::k_scale(0);
            ks[b][u] = D == 128 ? *reinterpret_cast<const uint16_t*>(sc + (u * 32 + lane) * 2)
                                : sc[u * 32 + lane];
          }
        if (!looked) look(m + 1);
        float s[U][NT][4];
        uint32_t sc[U][2][2];  // of keys g, g + 8: the scales of the lane's one or two groups
#pragma unroll
        for (int b = 0; b < U; ++b) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[b][nt][e] = 0.f;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x = e4m3_to_half(ks[b][u]);
            sc[b][u][0] = __byte_perm(x, x, 0x1010);
            sc[b][u][1] = D == 128 ? __byte_perm(x, x, 0x3232) : sc[b][u][0];
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          uint4 q[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) q[nt] = sm.q[qb][nt * kWords + w][lane];
#pragma unroll
          for (int b = 0; b < U; ++b) {
            uint32_t a[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              e2m1_to_half(kw[b][u][w], a[u]);
#pragma unroll
              for (int e = 0; e < 4; ++e) a[u][e] = half2_mul(a[u][e], sc[b][u][2 * w / kWords]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t f[4] = {a[0][2 * k], a[1][2 * k], a[0][2 * k + 1], a[1][2 * k + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16816(s[b][nt], f, k == 0 ? q[nt].x : q[nt].z, k == 0 ? q[nt].y : q[nt].w);
            }
          }
        }
        // Exponents, less the reference.
#pragma unroll
        for (int b = 0; b < U; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[b][nt][e] = fmaf(s[b][nt][e], c2[nt][e & 1], -ref[nt][e & 1]);
        if (key + 16 * U > min_lim || key + 16 * U > k_hi) {
#pragma unroll
          for (int b = 0; b < U; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int at = key + 16 * b + g + (e >> 1) * 8;
                if (at >= k_hi || at >= sm.lim[qb][nt * 8 + 2 * t + (e & 1)]) s[b][nt][e] = ninf;
              }
        }
        float over = ninf;
#pragma unroll
        for (int b = 0; b < U; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; e += 2) over = fmax3(over, s[b][nt][e], s[b][nt][e + 1]);
        if (j == 0 || __any_sync(0xffffffffu, over > kRescaleSlack + kHalfHeadroom)) {
          // The first scores, or some that outgrew the reference: every row's
          // moves to kHalfHeadroom below its maximum.  (A row that the first step's keys, the lowest,
          // are hidden from sees none of the later ones.)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float up = ninf;
#pragma unroll
              for (int b = 0; b < U; ++b) up = fmax3(up, s[b][nt][e], s[b][nt][e + 2]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, x));
              up -= kHalfHeadroom;
              if (up == ninf || (j > 0 && up < 0.f)) up = 0.f;
              const float alpha = j == 0 ? 1.f : ex2_approx(-up);
              ref[nt][e] += up;
              l[nt][e] *= alpha;
#pragma unroll
              for (int b = 0; b < U; ++b) s[b][nt][e] -= up, s[b][nt][e + 2] -= up;
#pragma unroll
              for (int mt = 0; mt < D / 16; ++mt) o[mt][nt][e] *= alpha, o[mt][nt][e + 2] *= alpha;
            }
        }
        uint32_t vw[U][2][kWords], vs[U][2];
#pragma unroll
        for (int b = 0; b < U; ++b)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            words(blk + b * Block::kBytes + Block::v_code(0, 0), u, vw[b][u]);
            vs[b][u] = *reinterpret_cast<const uint16_t*>(
                blk + b * Block::kBytes + Block::v_scale(D == 128 ? g : g / 2) + u * 8 + 2 * t);
          }
        __syncwarp();
        if (j + S < own) issue(j + S, c0);  // (this slot is free again)
        if (key + 16 * U > k_hi) {
          // Slots past the segment's keys may hold anything, and 0 * NaN is NaN.
#pragma unroll
          for (int b = 0; b < U; ++b)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int first = key + 16 * b + u * 8 + 2 * t;
              if (first >= k_hi) vs[b][u] = 0u;
              if (first + 1 >= k_hi) vs[b][u] &= 0xffu;
            }
        }
        uint32_t pt[U][NT][2], v[U][2];
#pragma unroll
        for (int b = 0; b < U; ++b) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = ex2_approx(s[b][nt][e]);
              l[nt][e & 1] += x[e];
            }
            pt[b][nt][0] = transpose_8x8(pack_f16x2(x[0], x[1]));
            pt[b][nt][1] = transpose_8x8(pack_f16x2(x[2], x[3]));
          }
          v[b][0] = e4m3_to_half(vs[b][0]);
          v[b][1] = e4m3_to_half(vs[b][1]);
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w)
#pragma unroll
          for (int b = 0; b < U; ++b) {
            uint32_t a[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              e2m1_to_half(vw[b][u][w], a[u]);
#pragma unroll
              for (int e = 0; e < 4; ++e) a[u][e] = half2_mul(a[u][e], v[b][u]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t f[4] = {a[0][2 * k], a[0][2 * k + 1], a[1][2 * k], a[1][2 * k + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816(o[2 * w + k][nt], f, pt[b][nt][0], pt[b][nt][1]);
            }
          }
      }
      if (lane == 0 && !fail) mbar_arrive(&sm.q_empty[qb]);
    }
    // ------------------------------------------------------ the unit's result
    // The next segment's first loads, before the warps wait for one another.
    // (Every warp comes to both votes, whatever failed, and all leave together.)
    const int was_end = end, r_rows = rows, r_tok0 = tok0, r_head0 = head0,
              r_slot = oslot;
    if (!was_end) take(m + 1);
    if (named_vote(1, 32 * W, fail) || was_end) break;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
        const int r = nt * 8 + 2 * t + e;
        if (g == 0) {
          sm.part_m[warp][r] = ref[nt][e];
          sm.part_l[warp][r] = l[nt][e];
        }
        // Channels g d/8 .. of the row: o[mt] holds 2 mt (its first half) and 2 mt + 1.
        if (r < r_rows)
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const int chunk = (g * (D / 32) + i) ^ t;
            *reinterpret_cast<float4*>(&sm.part_o[warp][r][chunk * 4]) =
                make_float4(o[2 * i][nt][e], o[2 * i][nt][e + 2], o[2 * i + 1][nt][e],
                            o[2 * i + 1][nt][e + 2]);
          }
      }
    named_bar_sync(1, 32 * W);
    for (int x = tid; x < r_rows * (D / 2); x += 32 * W) {  // a row to a warp (or half of one)
      const int r = x / (D / 2), ch = x % (D / 2) * 2;
      float2 y[W];
#pragma unroll
      for (int w = 0; w < W; ++w)
        y[w] = *reinterpret_cast<const float2*>(
            &sm.part_o[w][r][((ch >> 2) ^ ((r >> 1) & 3)) * 4 + (ch & 3)]);
      // Lane w (of every 16) weighs warp w's part.
      float pm = ninf, pl = 0.f;
      if ((lane & 15) < W) pm = sm.part_m[lane & 15][r], pl = sm.part_l[lane & 15][r];
      float top = pl == 0.f ? ninf : pm;
#pragma unroll
      for (int e = 8; e > 0; e >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
      const float weight = pl == 0.f ? 0.f : exp2f(pm - top);
      float sum = pl * weight;
#pragma unroll
      for (int e = 8; e > 0; e >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, e);
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = __shfl_sync(0xffffffffu, weight, w);
        acc.x += f * y[w].x, acc.y += f * y[w].y;
      }
      // (The values' scale by itself: over the sum it may be too small to hold.)
      const float own = sum == 0.f ? 0.f : 1.f / sum;
      acc.x = acc.x * own * p.v_scale, acc.y = acc.y * own * p.v_scale;
      const float lse2 = sum == 0.f ? ninf : top + log2f(sum);
      const int tok = r / p.G;
      const long long at = (long long)(r_tok0 + tok) * p.Hq + r_head0 + (r - tok * p.G);
      if (r_slot >= 0) {
        const long long row = ((long long)cta * 2 + r_slot) * ph.slot_rows + r;
        *reinterpret_cast<float2*>(ph.slot_o + row * D + ch) = acc;
        if (ch == 0) ph.slot_lse[row] = lse2;
      } else {
        *reinterpret_cast<uint32_t*>(p.o + at * D + ch) = pack_bf16x2(acc.x, acc.y);
        if (ch == 0) p.lse[at] = lse2 == ninf ? ninf : lse2 * kLn2;
      }
    }
  }
  // After a failure: the copies on their way have to land before the CTA exits.
  for (; c < issued; ++c) drain_wait(&sm.full[warp][c % S], (c / S) & 1);
}

}  // namespace fa
