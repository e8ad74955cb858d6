// fa_paged4_tiles.cuh -- the prompt kernel's producers over a cache held in 4 bits:
// the list's segments, the K and V tiles turned into fp16, and the rows of Q.
//
// A 128-key tile is eight blocks of fa_kv4.cuh; four warps, one on each quarter of
// the SM, make two blocks of each tile, K and V in turn: 8,192 numbers a warp in
// the 2,600 cycles that a step of the tensor core takes.  (A warp for K and one
// for V, beside the softmax warps of two of the quarters, took 7,800.)  A lane
// reads 16 bytes (d = 64: 8) of a block's codes at a time, a step ahead of those
// it converts, and stores 16 bytes of the tile at a time, in the layout that TMA
// would leave: [d / 64][128 keys][128 bytes], the 16-byte chunk c of row r at
// c ^ (r % 8).  Which lane stores which of its pieces first is chosen so that
// eight lanes meet eight chunks.
//
// Measured: 4 chunks of 1,024 rows over 4K keys, H_q 32, H_kv 8, d = 128: 242 us with the
// tile warps (992 TFLOP/s, tensor pipe active 46%), bound by them beside the softmax:
// their instructions share its schedulers, and any use of a loaded value right behind
// the load waits for it.  Hence the reads a step ahead, looked at only when stored
// (295 -> 256 us with registers enough for that), and a block's place found once for
// K and V (256 -> 242).
//
// There every tile is made 16 times, once for each unit of 256 rows.  Where a sequence
// has more than 1,024 rows of a head, paged4_expand makes each once, by the same
// functions, into the workspace, in the image that shared memory takes, so that one
// copy of 32 KB is a tile.  Where that holds for all of the kernel's sequences, it runs
// without tile warps: 187 us (1,284 TFLOP/s, tensor pipe active 64% of its 168 us; over
// the bf16 cache 170), of which the making takes 15 (67 MB written) and the merge 12.
#pragma once

#include <type_traits>

#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_paged.cuh"
#include "sm100_ptx.cuh"

namespace fa {

// Walks the CTA's range of the list and publishes its segments; load_q loads the
// query rows of those with keys.
template <int kRing, class Smem, class LoadQ>
__device__ __forceinline__ void paged4_produce_items(const PagedParams& p, const PagedPhase& ph,
                                                     Smem& sm, PagedWalk& walk, int cta, int ctas,
                                                     LoadQ&& load_q) {
  volatile int* abortf = &sm.abort_flag;
  PagedRec* const rec = reinterpret_cast<PagedRec*>(ph.rec + cta * kPagedRecBytes);
  bool ok = true;
  paged_walk_begin(p, ph, sm.scan, walk, cta, ctas);
  // Publishes the walk's next segment as item m; false at the list's end.
  auto publish = [&](int m) -> bool {
    const PagedItem it = paged_next(p, ph, walk, cta);
    const int is = m % kRing;
    if (m >= kRing)
      ok = mbar_wait(&sm.item_empty[is], (m / kRing - 1) & 1, p.status, abortf, kSitePgItemEmpty);
    ok = __all_sync(0xffffffffu, ok);
    if (ok && lane_id() == 0) {
      sm.item[is] = it;
      mbar_arrive(&sm.item_full[is]);
    }
    __syncwarp();
    return ok && !it.end;
  };
  bool more = publish(0);
  if (ok && lane_id() == 0) {
    if (more)
      *rec = paged4_first_rec(sm.item[0], walk);
    else
      rec->split = 0;
  }
  // Item m + 1 is known before item m's query rows have a place.
  for (int m = 0; more; ++m) {
    more = publish(m + 1);
    if (!ok) break;
    const PagedItem it = sm.item[m % kRing];  // (only this warp writes the records)
    if (it.nj > 0) ok = load_q(it);
    ok = __all_sync(0xffffffffu, ok);
    more = more && ok;
  }
  __syncwarp();
}

// What a lane has read of two blocks: its codes of K or V, and scales; of V how many
// keys the blocks hold (the scales of slots past them become 0: their codes may be
// anything, and are finite).
template <int D>
struct Raw4 {
  uint32_t code[2][2][D / 32];
  uint32_t scale[2][2];
  int keys;
};

// Reads two blocks (at blk[0] and blk[1]), keys in their slots until `keys` and `keys`
// - 16 of them.  Straight-line code that looks at nothing it loads.  (Ordinary loads: an
// append may write the blocks after this kernel has begun, up to its wait_prior_grid,
// which loads for data that stay the same while a kernel runs do not allow.)
template <int D, bool kV>
__device__ __forceinline__ void read_raw4(const uint8_t* const (&blk)[2], int keys, Raw4<D>& r) {
  using Block = Kv4Block<D>;
  const int lane = (int)lane_id(), g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint8_t* const codes = blk[b] + (kV ? Block::v_code(0, 0) : Block::k_code(0)) + lane * (D / 8);
    const uint8_t* const scales =
        blk[b] + (kV ? Block::v_scale(D == 128 ? g : g / 2) + 2 * t
                     : Block::k_scale(0) + lane * (D == 128 ? 2 : 1));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(codes + u * 512);
        r.code[b][u][0] = x.x, r.code[b][u][1] = x.y;
        r.code[b][u][D / 32 - 2] = x.z, r.code[b][u][D / 32 - 1] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(codes + u * 256);
        r.code[b][u][0] = x.x, r.code[b][u][1] = x.y;
      }
      if constexpr (kV)
        r.scale[b][u] = *reinterpret_cast<const uint16_t*>(scales + u * 8);
      else if constexpr (D == 128)
        r.scale[b][u] = *reinterpret_cast<const uint16_t*>(scales + u * 64);
      else
        r.scale[b][u] = scales[u * 32];
    }
  }
  if constexpr (kV) r.keys = keys;
}

// Turns them into rows 32 part .. 32 part + 31 of a tile (of kRows rows).
template <int D, bool kV, int kRows = kTile>
__device__ __forceinline__ void store_raw4(const Raw4<D>& r, int part, uint8_t* tile) {
  const int lane = (int)lane_id(), g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t bytes = r.scale[b][u];
      if (kV && r.keys < 32) {  // (the end of a unit's keys)
        const int n = r.keys - (16 * b + 8 * u + 2 * t);
        bytes &= n > 1 ? 0xffffu : n > 0 ? 0xffu : 0u;
      }
      const uint32_t s = e4m3_to_half(bytes);
      if constexpr (!kV) {
        // Key g of these eight, channels t d/4 ..: a word is a chunk of eight.
        const int row = 32 * part + 16 * b + 8 * u + g;
        // (Lanes of the second 64 channels take the words of their second group first.)
        const bool swap = D == 128 && (t >> 1) != 0;
        const uint32_t lo = __byte_perm(s, s, 0x1010), hi = D == 128 ? __byte_perm(s, s, 0x3232) : lo;
        const uint32_t s0 = swap ? hi : lo, s1 = swap ? lo : hi;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int w = swap ? i ^ 2 : i;
          const uint32_t code = swap ? r.code[b][u][D == 128 ? i ^ 2 : i] : r.code[b][u][i];
          uint32_t x[4];
          e2m1_to_half(code, x);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = half2_mul(x[e], i >= 2 ? s1 : s0);
          const int ch = D == 128 ? (t & 1) * 4 + w : 2 * t + w;
          *reinterpret_cast<uint4*>(tile + (D == 128 ? (t >> 1) * (kRows * 128) : 0) + row * 128 +
                                    ((ch ^ (row & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
        }
      } else {
        // Keys 2t and 2t + 1 of these eight, channels g d/8 ..: two words are a
        // chunk of eight of both.
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint32_t x[8];
          e2m1_to_half(r.code[b][u][2 * i], reinterpret_cast<uint32_t(&)[4]>(x[0]));
          e2m1_to_half(r.code[b][u][2 * i + 1], reinterpret_cast<uint32_t(&)[4]>(x[4]));
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = half2_mul(x[e], s);
          const int ch = D == 128 ? g * 2 + i : g;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // (Lanes of odd g store the odd key first.)
            const int key = k ^ (g & 1), row = 32 * part + 16 * b + 8 * u + 2 * t + key;
            const uint32_t sel = key ? 0x7632u : 0x5410u;
            *reinterpret_cast<uint4*>(tile + (ch >> 3) * (kRows * 128) + row * 128 +
                                      (((ch & 7) ^ (row & 7)) << 4)) =
                make_uint4(__byte_perm(x[0], x[1], sel), __byte_perm(x[2], x[3], sel),
                           __byte_perm(x[4], x[5], sel), __byte_perm(x[6], x[7], sel));
          }
        }
      }
    }
  }
}

// The tiles of long prompts' sequences in fp16, once for all units: a warp makes a
// quarter of a tile of K or V, as the prompt kernel's warps do, in the warp's part
// of shared memory, `stage`, from where it leaves in whole lines; in the order of the
// sequences, as far as the room goes.  n_min: the fewest rows of those sequences.
template <int D>
__device__ __forceinline__ void paged4_expand(const Paged4Params& p, int n_min, int w, int warps,
                                              uint8_t (&stage)[32 * D * 2]) {
  constexpr int kBytes = kTile * D * 2;
  const int lane = (int)lane_id();
  const long long cap = (long long)p.max_pages << p.page_shift;
  long long before = 0;  // tiles of the sequences that were looked at
  for (int b0 = 0; b0 < p.B; b0 += 128) {  // four neighbours to a lane: their loads together
    int t0[4], t1[4], len[4], tiles[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = b0 + 4 * lane + i;
      t0[i] = t1[i] = len[i] = 0;
      if (b < p.B) t0[i] = p.cu_q[b], t1[i] = p.cu_q[b + 1], len[i] = p.seq_lens[b];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool on = paged_range_ok(t0[i], t1[i], p.T) && t1[i] - t0[i] >= n_min && len[i] > 0 &&
                      len[i] <= cap;
      tiles[i] = on ? min((len[i] - 1) / kTile + 1, p.expand + 1) : 0;  // (more have no room)
      sum += tiles[i];
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    long long at0 = before + upto - sum;
    int start[4];  // (-1: no room)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      start[i] = tiles[i] > 0 && at0 + tiles[i] <= p.expand ? (int)at0 : -1;
      at0 += tiles[i];
      if (w == 0 && b0 + 4 * lane + i < p.B) p.tile_base[b0 + 4 * lane + i] = start[i];
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      auto pick = [&](const int (&x)[4]) { return i == 0 ? x[0] : i == 1 ? x[1] : i == 2 ? x[2] : x[3]; };
      const int my_start = pick(start), my_tiles = pick(tiles), my_len = pick(len);
      for (unsigned left = __ballot_sync(0xffffffffu, my_start >= 0); left != 0; left &= left - 1) {
        const int src = __ffs(left) - 1, base = __shfl_sync(0xffffffffu, my_start, src);
        const int n = __shfl_sync(0xffffffffu, my_tiles, src) * p.Hkv * 8;
        const int keys = __shfl_sync(0xffffffffu, my_len, src);
        const int* const list = p.page_table + (long long)(b0 + 4 * src + i) * p.max_pages;
        const int at = (int)((long long)base * p.Hkv * 8 % warps);
        for (int x = w >= at ? w - at : w - at + warps; x < n; x += warps) {
          const int part = x & 3, tile = (x >> 3) / p.Hkv, h = (x >> 3) - tile * p.Hkv;
          const bool is_v = (x & 4) != 0;
          const int first = tile * kTile + 32 * part, key = first + 16 * (lane & 1);
          const int page = key < keys ? list[key >> p.page_shift] : 0;
          const bool valid = (unsigned)page < (unsigned)p.num_pages;
          if (!valid) {
            int abort_flag = 0;
            report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPage);
          }
          const unsigned long long mine = reinterpret_cast<unsigned long long>(
              p.pages + kv4_block_at(valid ? page : 0, p.Hkv, h, p.page_shift,
                                     key & (p.page_size - 1), Kv4Block<D>::kBytes));
          const uint8_t* blk[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            blk[e] = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, mine, e));
          uint8_t* const dst = p.tiles + ((long long)(base + tile) * p.Hkv + h) * (2 * kBytes) +
                               (is_v ? kBytes : 0);
          Raw4<D> raw;
          auto make = [&](auto v) {
            read_raw4<D, decltype(v)::value>(blk, keys - first, raw);
            if (lane == 0) bulk_wait_group_read0();  // (the last quarter has left)
            __syncwarp();
            store_raw4<D, decltype(v)::value, 32>(raw, 0, stage);
          };
          if (is_v)
            make(std::true_type{});
          else
            make(std::false_type{});
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int e = 0; e < D / 64; ++e)  // 64 channels
              bulk_store(dst + (e * kTile + 32 * part) * 128, stage + e * 4096, 4096);
            bulk_commit_group();
          }
          __syncwarp();
        }
      }
    }
  }
  if (lane == 0) bulk_wait_group0();
  __syncwarp();
}

// The warp that loads the tiles of the CTA's segments where all of them are in fp16.
// (A sequence that was left out, for its table's sake, takes what is there.)
template <int D, int S, int kRing, class Smem>
__device__ __forceinline__ void paged4_load_tiles(const Paged4Params& p, Smem& sm) {
  constexpr int kBytes = kTile * D * 2;
  volatile int* abortf = &sm.abort_flag;
  const int lane = (int)lane_id();
  bool ok = true;
  int c = 0;
  for (int m = 0; ok; ++m) {
    const int is = m % kRing;
    ok = mbar_wait(&sm.item_full[is], (m / kRing) & 1, p.status, abortf, kSitePgItemFull);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const PagedItem& it = sm.item[is];
    const int nj = it.nj, h = it.h, at = it.key / kTile;
    const bool end = it.end != 0;
    const int base = end ? 0 : p.tile_base[it.b];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[is]);
    if (end) break;
    for (int j = 0; ok && j < nj; ++j) {
      const int tile = base + at + j;
      const uint8_t* const src =
          p.tiles + ((long long)(base >= 0 && tile < p.expand ? tile : 0) * p.Hkv + h) * (2 * kBytes);
      for (int v = 0; ok && v < 2; ++v, ++c) {
        if (c >= S)
          ok = mbar_wait(&sm.kv_empty[c % S], (c / S - 1) & 1, p.status, abortf, kSitePgKvEmpty);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.kv_full[c % S], kBytes);
          bulk_load(sm.kv[c % S], src + v * kBytes, kBytes, &sm.kv_full[c % S]);
        }
        __syncwarp();
      }
    }
  }
  // After a failure: the copies on their way have to land before the CTA exits.
  if (*abortf && lane == 0)
    for (int x = max(0, c - S); x < c; ++x) drain_wait(&sm.kv_full[x % S], (x / S) & 1);
  __syncwarp();
}

// One of the warps that make the tiles of the CTA's segments: part `part` of each.
template <int D, int S, int kRing, class Smem>
__device__ __forceinline__ void paged4_produce_tiles(const Paged4Params& p, Smem& sm, int part) {
  volatile int* abortf = &sm.abort_flag;
  const int lane = (int)lane_id();
  bool ok = true;
  // The tile that is read next: its segment's place, its two blocks, and the pages of
  // the next tile's blocks (even lanes the first, odd lanes the second).  A block
  // past the keys, or without a page, reads page 0.
  // (Or, where the sequence's tiles are in fp16 already, blk[0]: this one's K, with V
  // behind it.)
  constexpr int kBytes = kTile * D * 2;
  int m = -1, left = 0, h = 0, key = 0, k_hi = 0, next = 0;
  bool end = false, whole = false;
  const int* list = nullptr;
  const uint8_t* blk[2] = {p.pages, p.pages};
  auto pages = [&](int first) -> int {
    const int at = first + 16 * (2 * part + (lane & 1));
    return at < k_hi ? list[at >> p.page_shift] : 0;
  };
  auto locate = [&](int page) {
    const bool valid = (unsigned)page < (unsigned)p.num_pages;
    const int at = key + 16 * (2 * part + (lane & 1));
    if (!valid) {
      int abort_flag = 0;
      report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPage);
    }
    const unsigned long long mine = reinterpret_cast<unsigned long long>(
        p.pages + kv4_block_at(valid ? page : 0, p.Hkv, h, p.page_shift, at & (p.page_size - 1),
                               Kv4Block<D>::kBytes));
#pragma unroll
    for (int b = 0; b < 2; ++b)
      blk[b] = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, mine, b));
  };
  auto step = [&] {
    if (--left > 0) {
      key += kTile;
      if (whole) {
        blk[0] += 2ll * kBytes * p.Hkv;
        return;
      }
      const int page = next;
      next = left > 1 ? pages(key + kTile) : 0;
      locate(page);
      return;
    }
    do {  // the next segment with keys
      const int is = ++m % kRing;
      ok = mbar_wait(&sm.item_full[is], (m / kRing) & 1, p.status, abortf, kSitePgItemFull);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const PagedItem& it = sm.item[is];
      end = it.end != 0;
      left = it.nj, h = it.h, key = it.key, k_hi = it.k_hi;
      list = p.page_table + (long long)it.b * p.max_pages;
      const int base = p.expand > 0 && !end ? p.tile_base[it.b] : -1;
      whole = base >= 0;
      if (whole) blk[0] = p.tiles + ((long long)(base + key / kTile) * p.Hkv + h) * (2 * kBytes);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[is]);
    } while (!end && left == 0);
    if (end || whole) return;
    const int page = pages(key);
    next = left > 1 ? pages(key + kTile) : 0;
    locate(page);
  };
  auto ready = [&](int c) -> bool {
    if (c >= S)
      ok = mbar_wait(&sm.kv_empty[c % S], (c / S - 1) & 1, p.status, abortf, kSitePgKvEmpty);
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };
  auto hand_on = [&](int c) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.kv_full[c % S]);
  };
  // Slot c from a tile in fp16: one warp copies it, the others only hand it on.
  int copied = 0;  // tiles up to the last one copied
  auto copy = [&](int c, const uint8_t* src) {
    if (lane == 0) {
      if (part == 0) {
        mbar_arrive_expect_tx(&sm.kv_full[c % S], kBytes);
        bulk_load(sm.kv[c % S], src, kBytes, &sm.kv_full[c % S]);
      } else {
        mbar_arrive(&sm.kv_full[c % S]);
      }
    }
    __syncwarp();
    copied = c + 1;
  };
  Raw4<D> k, v;
  step();
  if (ok && !end && !whole) {
    read_raw4<D, false>(blk, 0, k);
    read_raw4<D, true>(blk, k_hi - (key + 32 * part), v);
  }
  for (int c = 0; ok && !end; c += 2) {
    const uint8_t* const src = whole ? blk[0] : nullptr;
    if (!ready(c)) break;
    if (src != nullptr) {
      copy(c, src);
    } else {
      store_raw4<D, false>(k, part, sm.kv[c % S]);
      hand_on(c);
    }
    step();
    if (!ok) break;
    const bool raw = !end && !whole;
    if (raw) read_raw4<D, false>(blk, 0, k);
    if (!ready(c + 1)) break;
    if (src != nullptr) {
      copy(c + 1, src + kBytes);
    } else {
      store_raw4<D, true>(v, part, sm.kv[(c + 1) % S]);
      hand_on(c + 1);
    }
    if (raw) read_raw4<D, true>(blk, k_hi - (key + 32 * part), v);
  }
  // After a failure: the copies on their way have to land before the CTA exits.
  if (*abortf && part == 0 && lane == 0)
    for (int c = max(0, copied - S); c < copied; ++c) drain_wait(&sm.kv_full[c % S], (c / S) & 1);
  __syncwarp();
}

// Row r of a Q tile from bf16 to fp16, in place, times the power of two that takes
// it to fp16's range; returns the factor from products to exponents (c2 that of
// the row as it was), which is never 0: what vanishes is a tiny one, negative where
// the kernel's form is that of negative scales (c2 may be a 0 of either sign, its
// product with the keys' scale being too small to hold).
template <int D, bool kNeg>
__device__ __forceinline__ float q_row_to_half(uint8_t* tile, int r, float c2) {
  uint8_t* const row = tile + r * 128;
  uint32_t top = 0u;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {  // (in an order of chunks that meets every bank)
    const uint4 x =
        *reinterpret_cast<const uint4*>(row + (c >> 3) * (kTile * 128) + ((c ^ r) & 7) * 16);
    top = kv4_top(kv4_top(kv4_top(kv4_top(top, x.x), x.y), x.z), x.w);
  }
  const int e = kv4_row_exponent(top);
  const float f = kv4_pow2(e);
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    uint4* const at = reinterpret_cast<uint4*>(row + (c >> 3) * (kTile * 128) + ((c ^ r) & 7) * 16);
    const uint4 x = *at;
    auto turn = [&](uint32_t w) {
      uint32_t y;
      asm("cvt.rn.f16x2.f32 %0, %1, %2;"
          : "=r"(y)
          : "f"(__uint_as_float(w & 0xffff0000u) * f), "f"(__uint_as_float(w << 16) * f));
      return y;
    };
    *at = make_uint4(turn(x.x), turn(x.y), turn(x.z), turn(x.w));
  }
  const float x = c2 * kv4_pow2(-e), tiny = 1.17549435e-38f;
  return fabsf(x) >= tiny ? x : (kNeg ? -tiny : tiny);
}

}  // namespace fa
