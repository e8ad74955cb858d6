// fa_internal.h -- declarations shared by the C-ABI front end (fa_api.cu)
// and the kernels (fa_fwd.cu, fa_bwd.cu).  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/fa.h"

namespace fa {

constexpr int kTile = 128;        // rows of a Q tile and of a K/V tile
constexpr int kPairRows = 2 * kTile;  // query rows of one forward work item
constexpr int kHeadGroup = 8;     // heads whose work items are kept together

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Number of 128-key tiles query tile `qt` (rows 128*qt .. 128*qt+127) visits.
__host__ __device__ inline int fwd_kv_tiles(int qt, int n_kv, int causal) {
  if (!causal) return n_kv;
  const int last = qt + 1;  // keys j <= row: tiles 0 .. qt
  return last < n_kv ? last : n_kv;
}

// The forward kernel's work order.  Items are (head, pair of query tiles).
// Heads are taken in groups of kHeadGroup so that the CTAs running at the
// same time share few heads' K/V in L2; inside a group the pairs go from
// the last (most keys under a causal mask) to the first, so under a causal
// mask the longest items start first and the short ones fill the tail.
__host__ __device__ inline void fwd_item(int t, int BH, int n_pairs, int* bh, int* pair) {
  const int per_group = kHeadGroup * n_pairs;
  const int g = t / per_group;
  const int gsize = (BH - g * kHeadGroup) < kHeadGroup ? (BH - g * kHeadGroup) : kHeadGroup;
  const int idx = t - g * per_group;
  *pair = n_pairs - 1 - idx / gsize;
  *bh = g * kHeadGroup + idx % gsize;
}

// Forward parameters.  The general form has H_q query heads sharing H_kv
// K/V heads in groups of G = H_q / H_kv; the G * N_q query rows of one K/V
// head are contiguous in a [B][H_q][N_q][d] array, so the kernel treats them
// as one packed row space of `rows` rows per K/V head.  Row r is query
// position r % N_q.  The square entry point is G = 1, N_q = N_kv = N.
struct FwdParams {
  void* o;           // [BH][rows][d] bf16
  float* lse;        // [BH][rows] fp32
  float* o_part;     // splits > 1: [splits][BH][rows][d] fp32, each split's O
  float* lse_part;   // splits > 1: [splits][BH][rows] fp32, each split's lse
  const uint8_t* block_mask;  // optional [n_kv][n_kv] 0/1 over (query tile, key tile)
  const float* fp8_amax;      // FP8 forward: [3][BH] amax of the (rotated) Q, K and of V
  int fp8_hadamard;           // FP8 forward: Q and K were rotated by H_d
  int* status;       // device status word (2 ints: code, site)
  int BH;            // B * H_kv
  int rows;          // packed query rows per K/V head: G * N_q
  int Nq;            // query positions per query head
  int Nkv;           // keys per K/V head
  int causal_off;    // N_kv - N_q: query i sees keys j <= i + causal_off
  int n_kv;          // ceil(N_kv / 128)
  int n_pairs;       // ceil(rows / 256)
  int splits;        // key splits (1: O and lse written directly)
  int tiles_per_split;
  int causal;
  float scale_log2;  // scale * log2(e)
  int grid;          // CTAs launched
  // Dynamic item claiming (persistent CTAs under a causal or block mask):
  // {items claimed, CTAs finished}, zero at launch; the last CTA to finish
  // sets both back to zero.  Null: the static split of the list.
  int* sched;
};

// Slots of the forward's work counters: calls on one stream share a slot
// (they run in order), calls on different streams get different slots.
constexpr int kFwdSchedSlots = 64;
constexpr int kFwdSchedStride = 32;  // ints per slot: one 128-byte line each

// Number of 128-key tiles, counted from key 0, that the query rows
// [r0, min(r0 + 128, rows)) of a K/V head need: all of them without a mask,
// else up to the last key visible to the row with the largest position.
__host__ __device__ inline int fwd_tile_key_tiles(int r0, const FwdParams& p) {
  if (r0 >= p.rows) return 0;
  if (!p.causal) return p.n_kv;
  const int len = (r0 + kTile < p.rows ? r0 + kTile : p.rows) - r0;
  const int i0 = r0 % p.Nq;
  const int maxi = (i0 + len - 1 >= p.Nq) ? p.Nq - 1 : i0 + len - 1;
  long long lim = (long long)maxi + p.causal_off + 1;
  if (lim <= 0) return 0;
  if (lim > p.Nkv) lim = p.Nkv;
  return ceil_div((int)lim, kTile);
}

// CTA that runs work item `idx` of a longest-first list on `ctas` persistent
// CTAs: round k = idx / ctas is taken in order when k is even and in
// reverse when k is odd ("snake" order).
__host__ __device__ inline int snake_cta(int idx, int ctas) {
  const int k = idx / ctas, pos = idx % ctas;
  return (k & 1) ? ctas - 1 - pos : pos;
}

// The forward kernel's grid.  Without a mask every item costs the same and
// min(items, SMs) persistent CTAs split the list statically.  Under a causal
// mask item costs differ by up to N/128, so a static split cannot balance
// them: the CTAs take the longest-first list greedily instead (the LPT
// rule).  With a work counter (FwdParams::sched) min(items, SMs) persistent
// CTAs claim the items in list order as they become ready for one; without
// one every item gets its own CTA and the hardware hands CTAs to SMs in
// list order as SMs free up.  This function gives the grid of the latter.
__host__ __device__ inline int fwd_grid(int BH, int n_pairs, int causal, int sm_count) {
  const long long items = (long long)BH * n_pairs;
  if (causal) return (int)items;
  return (int)(items < sm_count ? items : sm_count);
}

struct BwdParams {
  const void* o;     // [BH][N][d] bf16 (forward output)
  const void* dout;  // [BH][N][d] bf16
  const float* lse;  // [BH][N] fp32
  void* dq;          // [BH][N][d] bf16
  void* dk;
  void* dv;
  float* dq_acc;     // workspace: [BH][n_kv*128][d] fp32, tile-blocked
  float* delta;      // workspace: [BH][n_kv*128] fp32 (-D_i)
  float* lse2;       // workspace: [BH][n_kv*128] fp32 (-lse_i * log2 e, -inf past N)
  int* status;
  const uint8_t* block_mask;  // optional [n_kv][n_kv] 0/1 over (query tile, key tile)
  int BH, N;
  int n_kv;
  int causal;
  float scale;
  float scale_log2;
  int* sched;    // workspace: the main kernel's work-item counter (zeroed by prep)
  int sm_count;  // persistent grid size of the main kernel
};

// Build a rank-3 tensor map over a [BH][N][d] bf16 array: dims (d, N, BH),
// box (64, 128, 1), 128-byte swizzle, zero fill outside.  Returns 0 or an
// FA_ERR_* code.
int make_tmap_bhnd(const void* base, int BH, int N, int d, CUtensorMap* out);

// The same map with a box of `box_rows` rows (the pair kernel's K halves).
int make_tmap_bhnd_rows(const void* base, int BH, int N, int d, int box_rows, CUtensorMap* out);

// The forward pass on CTA pairs (tcgen05 cta_group::2): square shapes with
// d = 128 and no mask.  tkh is K's map with a 64-row box.  At most
// `max_pairs` pairs are launched (fwd_pair_max_active: pairs that fit at once).
int launch_fwd_pair(const CUtensorMap& tq, const CUtensorMap& tkh, const CUtensorMap& tv,
                    const FwdParams& p, cudaStream_t stream, int max_pairs);
int fwd_pair_max_active(int sm_count);

// `to` is a tensor map over O with the shape of tq's; only the square bf16
// kernels that stage O for TMA stores use it.
int launch_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
               const CUtensorMap& to, const FwdParams& p, int d, cudaStream_t stream);

// Byte offsets of the general forward pass's split workspace: each split's
// fp32 O, then each split's lse, 256-byte aligned.
struct FwdWorkspace {
  size_t o_part, lse_part, total;
};
inline FwdWorkspace fwd_workspace_layout(long long splits, long long BH, long long rows, int d) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  FwdWorkspace w;
  w.o_part = 0;
  w.lse_part = up((size_t)(splits * BH * rows) * (size_t)d * sizeof(float));
  w.total = w.lse_part + up((size_t)(splits * BH * rows) * sizeof(float));
  return w;
}

// Byte offsets of the backward workspace's parts for these sizes:
// the fp32 dQ accumulator, then -D, then -lse * log2(e), then the main
// kernel's work-item counter (one int in a 256-byte slot), each 256-byte
// aligned.
struct BwdWorkspace {
  size_t dq_acc, delta, lse2, sched, total;
};
inline BwdWorkspace bwd_workspace_layout(long long BH, int N, int d) {
  const size_t rows = (size_t)BH * (size_t)ceil_div(N, kTile) * kTile;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  BwdWorkspace w;
  w.dq_acc = 0;
  w.delta = up(rows * (size_t)d * sizeof(float));
  w.lse2 = w.delta + up(rows * sizeof(float));
  w.sched = w.lse2 + up(rows * sizeof(float));
  w.total = w.sched + 256;
  return w;
}

// Byte offsets of the FP8 forward pass's workspace (d = 128): the E4M3
// codes of the (rotated) Q and K, [BH][N][d]; the codes of V transposed per
// head, [BH][d][n_kv * 128] (keys past N are code 0); then the per-head
// absolute maxima of Q, K and V, [3][BH] fp32.  Parts 256-byte aligned.
struct Fp8Workspace {
  size_t q8, k8, vt8, amax, total;
};
inline Fp8Workspace fp8_workspace_layout(long long BH, int N, int d) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t qk = (size_t)BH * (size_t)N * (size_t)d;
  const size_t vt = (size_t)BH * (size_t)d * (size_t)ceil_div(N, kTile) * kTile;
  Fp8Workspace w;
  w.q8 = 0;
  w.k8 = up(qk);
  w.vt8 = w.k8 + up(qk);
  w.amax = w.vt8 + up(vt);
  w.total = w.amax + up((size_t)3 * BH * sizeof(float));
  return w;
}

// Quantise bf16 Q, K, V ([BH][N][128]) into the FP8 workspace `ws` laid out
// by fp8_workspace_layout; with `hadamard` the rows of Q and K are first
// multiplied by the 128 x 128 Sylvester Hadamard matrix.
int launch_fp8_quantize(const void* q, const void* k, const void* v, int BH, int N, int hadamard,
                        char* ws, const Fp8Workspace& layout, cudaStream_t stream);

// The paged key/value cache (fa_kv_append, fa_fwd_paged): packed rows
// [T][heads][d], pages [num_pages][Hkv][page_size][d].
struct KvAppendParams {
  const __nv_bfloat16* q;  // null: no queries
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_pages;
  __nv_bfloat16* v_pages;
  const int* page_table;  // [B][max_pages]
  const int* seq_lens;    // [B], new tokens included
  const int* cu_q;        // [B + 1]
  const float* rope;      // [rope_len][rope_dim]: cosines, then sines (rope_dim / 2 each)
  int* status;
  int T, B, Hq, Hkv;
  long long q_stride, k_stride, v_stride, q_out_stride;  // elements between rows
  int num_pages, page_size, page_shift, max_pages;
  int rope_dim, rope_len, interleaved;
};
int launch_kv_append(const KvAppendParams& p, int d, cudaStream_t stream);

// CTAs that share a call's work at most (one per SM; GB300 has 152), which
// sizes the workspace without a device.
constexpr int kPagedMaxCtas = 160;
// Most query rows of a unit in the decode kernel; a unit of the prompt kernel has
// kPairRows (two 128-row Q tiles).
constexpr int kPagedDecodeRows = 64;

struct PagedParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_pages;
  const __nv_bfloat16* v_pages;
  __nv_bfloat16* o;  // [T][Hq][d]
  float* lse;        // [T][Hq]
  const int* page_table;
  const int* seq_lens;
  const int* cu_q;
  const int* prefix_pages;  // null: no shared prefix
  int* status;
  int T, B, Hq, Hkv, G;
  long long q_stride;
  int num_pages, page_size, page_shift, max_pages;
  int prefix_len;
  int max_q;
  int causal;
  float scale_log2;
  int ctas;         // persistent CTAs
  char* workspace;  // PagedWorkspace
};

// How a call runs.  rows: of a unit in the attention of the sequences' own keys
// (8, 16, 32 or 64: the decode kernel; 256: the prompt kernel); prefix_rows: in
// that of the shared prefix by the rows of the whole batch.
//
// In a batch of long and short sequences, those of up to small_rows rows go to
// the decode kernel and the others to the prompt kernel, whose Q tiles a
// decoding sequence leaves almost empty (30 decoding sequences and two chunks
// of 500 tokens took 88 us on the prompt kernel alone).  A batch counts as
// mixed when its rows are fewer than a prompt unit per sequence on average but
// max_q says that one sequence has more than a decode unit, unless max_q makes
// all of them equal.
//
// duo: a prompt and a decode kernel side by side in one launch (for decode
// units of at most 16 rows): the two kinds of a mixed batch, or the prefix and
// the sequences' own keys when these are the decode kernel's, joined by a warp
// per row, which pays up to some ten thousand rows.
struct PagedForm {
  int rows, small_rows, share, prefix_rows, duo;
};
inline int paged_unit_rows(long long rows) {
  return rows <= 8 ? 8 : rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= kPagedDecodeRows ? 64 : kPairRows));
}
inline PagedForm paged_form(int T, int B, int Hq, int G, int max_q, int prefix_len) {
  PagedForm f;
  f.rows = paged_unit_rows((long long)(max_q < T ? max_q : T) * G);
  f.small_rows = 0;
  if (f.rows == kPairRows && B > 1 && G <= kPagedDecodeRows &&
      (long long)T * G < (long long)kPairRows * B && (long long)B * max_q > T)
    f.small_rows = paged_unit_rows(G);
  f.share = prefix_len > 0 ? 1 : 0;
  f.prefix_rows = paged_unit_rows((long long)T * G);
  if (f.share)
    f.duo = f.rows <= 16 && f.prefix_rows == kPairRows && (long long)T * Hq <= 16384;
  else
    f.duo = f.small_rows > 0 && f.small_rows <= 16;
  return f;
}

// Byte offsets of the paged forward's workspace, 256-byte aligned: for each of
// two phases of a call the split records of the CTAs and their partial results
// (two slots each: fp32 O rows, then the rows' logsumexp); with a shared prefix
// its results, fp32 [T][Hq][d] and [T][Hq]; in a duo the phases' CTA counts,
// and with a prefix the results of the sequences' own keys and which slots hold
// the parts of each phase's units (8 bytes a token and key/value head).
struct PagedWorkspace {
  size_t rec[2], slot_o[2], slot_lse[2], pre_o, pre_lse, own_o, own_lse, parts[2], ctas, total;
};
constexpr size_t kPagedRecBytes = 64;
inline PagedWorkspace paged_workspace_layout(int T, int Hq, int Hkv, int d, const PagedForm& f) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  int rows[2] = {f.rows, f.small_rows};
  if (f.share && f.duo) {
    rows[0] = f.prefix_rows;
    rows[1] = f.rows;
  } else if (f.share && f.prefix_rows > f.rows) {
    rows[0] = f.prefix_rows;
  }
  PagedWorkspace w;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up(bytes);
    return here;
  };
  for (int k = 0; k < 2; ++k) {
    const size_t slots = (size_t)kPagedMaxCtas * 2 * (size_t)rows[k];
    w.rec[k] = take(rows[k] > 0 ? kPagedMaxCtas * kPagedRecBytes : 0);
    w.slot_o[k] = take(slots * (size_t)d * sizeof(float));
    w.slot_lse[k] = take(slots * sizeof(float));
  }
  const size_t pre = f.share ? (size_t)T * (size_t)Hq : 0, own = f.duo ? pre : 0;
  w.pre_o = take(pre * (size_t)d * sizeof(float));
  w.pre_lse = take(pre * sizeof(float));
  w.own_o = take(own * (size_t)d * sizeof(float));
  w.own_lse = take(own * sizeof(float));
  for (int k = 0; k < 2; ++k) w.parts[k] = take(own > 0 ? (size_t)T * (size_t)Hkv * 8 : 0);
  w.ctas = take(f.duo ? 2 * sizeof(int) : 0);
  w.total = at;
  return w;
}

int launch_fwd_paged(const PagedParams& p, int d, cudaStream_t stream);

// A rank-3 tensor map over packed rows [T][heads][d] bf16 with `stride`
// elements between rows: dims (d, heads, T), box (64, box_heads, box_rows),
// 128-byte swizzle, zero fill outside.
int make_tmap_rows(const void* base, int heads, int T, long long stride, int d, int box_heads,
                   int box_rows, CUtensorMap* out);

// A rank-3 tensor map over a [BH][rows][inner] array of bytes: box
// (128, 128, 1), 128-byte swizzle, zero fill outside.
int make_tmap_u8(const void* base, int BH, int rows, int inner, CUtensorMap* out);

// phase_mask: bit 0 prep, bit 1 main, bit 2 convert.
int launch_bwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
               const CUtensorMap& tdo, const BwdParams& p, int d, cudaStream_t stream,
               int phase_mask);

}  // namespace fa
