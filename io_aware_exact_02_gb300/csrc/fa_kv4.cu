// fa_kv4.cu -- appending new keys and values to a paged cache held in 4 bits,
// with the rotary position embedding of the new queries and keys applied on the
// way, and reading rows of it back.
//
// Rows, positions and the rotation are those of fa_kv.cu; the numbers and their
// layout those of fa_kv4.cuh.  The rotated keys are quantised from fp32, each
// product and difference of the rotation rounded by itself, so that a code does
// not depend on how the compiler joins them.
//
// 16,384 rows of 32 query and 8 key/value heads, d = 128: append 69 us (5.1 TB/s of the
// 6.8 that a copy reaches; keys and values alone 34 us), reading back 19 us (4.5 TB/s).
// Neither the issue slots (58% and 52%) nor memory are full: of the 12 cycles that a
// warp takes for an instruction it waits 6 for loads from global memory.  Twice as many
// registers a thread, two rows to find a place for at a time, made the append 106 us.
//
// A byte of V holds a pair of neighbouring keys.  The row of the even slot
// writes both where the odd slot's row is new too; a row whose neighbour is not
// new keeps that one's half.
#include <cuda_bf16.h>

#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_paged.cuh"
#include "fa_rope.cuh"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ void widen8(const uint4& x, float* y) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = bf2(w[i]);
    y[2 * i] = a.x;
    y[2 * i + 1] = a.y;
  }
}

// (a, b) turned by the angle of cosine c and sine s.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  b = __fadd_rn(__fmul_rn(x, s), __fmul_rn(y, c));
}

__device__ __forceinline__ float top8(const float* y) {
  float m = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(y[i]));
  return m;
}

// Infinities (of a group whose largest magnitude is one) to numbers beyond every
// code's, for kv4_quotient.
template <int N>
__device__ __forceinline__ void bound(float (&y)[N], float top) {
  if (top != __int_as_float(0x7f800000)) return;
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = fminf(fmaxf(y[i], -65536.f), 65536.f);
}

// Half of a value row's group, divided by the tensor's scale.
__device__ __forceinline__ void scaled8(const uint4& x, float inv, float (&y)[8]) {
  widen8(x, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(y[i], inv);
}
// The largest magnitude of a group.
__device__ __forceinline__ float top16(const uint4 (&x)[2], float inv) {
  float y[8];
  scaled8(x[0], inv, y);
  const float t = top8(y);
  scaled8(x[1], inv, y);
  return max_nan(t, top8(y));
}
// Half of a group's quotients.
__device__ __forceinline__ void quotients8(const uint4& x, float inv, float top, float s, float r,
                                           float (&y)[8]) {
  scaled8(x, inv, y);
  bound(y, top);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = kv4_quotient(y[i], s, r);
}

// Where a row goes: its sequence, position, and page (b -1: nowhere).
struct RowPlace {
  int b, pos, t0, t1, page;  // t0, t1: the sequence's rows
};

// The place of row t.  `last`: that of row t - 1, if the CTA has had it (b -1: not):
// the next row of the same sequence needs no search, and mostly the same page.
template <class Params>
__device__ __forceinline__ RowPlace place_row(const Params& p, int t, const RowPlace& last,
                                              int rope_len) {
  RowPlace r = last;
  int abort_flag = 0;
  if (last.b >= 0 && t < last.t1) {
    ++r.pos;
  } else {
    const PagedRow at = paged_row(p.cu_q, p.seq_lens, p.B, p.T, t, p.status);
    r.b = at.b;
    r.pos = at.pos;
    r.page = -1;
    if (at.b < 0) return r;
    r.t0 = p.cu_q[at.b];
    r.t1 = p.cu_q[at.b + 1];
  }
  if (r.pos < 0 || r.pos >= (long long)p.max_pages << p.page_shift ||
      (rope_len >= 0 && r.pos >= rope_len)) {
    if (threadIdx.x == 0) report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPosition);
    r.b = -1;
    return r;
  }
  if (r.page < 0 || (r.pos & (p.page_size - 1)) == 0)
    r.page = p.page_table[(long long)r.b * p.max_pages + (r.pos >> p.page_shift)];
  if (r.page < 0 || r.page >= p.num_pages) {
    if (threadIdx.x == 0) report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPage);
    r.b = -1;
  }
  return r;
}

// The ranges of all sequences, those without a row among them, by the threads of
// all CTAs in turn.
template <class Params>
__device__ __forceinline__ void check_ranges(const Params& p) {
  for (long long b = (long long)blockIdx.x * kThreads + threadIdx.x; b < p.B;
       b += (long long)gridDim.x * kThreads) {
    int abort_flag = 0;
    if (!paged_range_ok(p.cu_q[b], p.cu_q[b + 1], p.T))
      report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedRows);
  }
}

// Row t, threads as in fa_kv.cu: a thread owns two 8-channel chunks of every kRows-th
// head.
template <int D>
__device__ __forceinline__ void append_row(const Kv4AppendParams& p, int t, const RowPlace& at) {
  using Block = Kv4Block<D>;
  constexpr int kPairs = D / 16;             // chunk pairs (and groups) of a head
  constexpr int kRows = kThreads / kPairs;   // heads in one sweep of the CTA
  const int pr = threadIdx.x % kPairs, row = threadIdx.x / kPairs;
  const int rd = p.rope_dim, half = rd / 16;  // chunks that are first halves
  int ca = 2 * pr, cb = 2 * pr + 1;
  bool turn = false;
  if (p.interleaved) {
    turn = ca * 8 < rd;
  } else if (pr < half) {
    ca = pr;
    cb = pr + half;
    turn = true;
  }
  const int page = at.page;
  // (Read where it is used, from L1 but for the first time: to keep the 16 numbers
  // through the values' quantisation takes registers that it has not.)
  const float* const tab = p.rope + (long long)at.pos * rd + pr * 8;
  const int slot = at.pos & (p.page_size - 1), r = slot & 15;
  const int Hq = p.q ? p.Hq : 0;
  const bool odd = (r & 1) != 0;
  // (A next row past the rotation's table is refused: it writes nothing, nor does this one for it.)
  const bool before = odd && t > at.t0,
             after = !odd && t + 1 < at.t1 && (rd == 0 || at.pos + 1 < p.rope_len);
  const unsigned group = (kPairs == 8 ? 0xffu : 0xfu) << ((threadIdx.x & 31) & ~(kPairs - 1));
  for (int h = row; h < Hq + 2 * p.Hkv; h += kRows) {
    if (h < Hq) {
      const __nv_bfloat16* src = p.q + t * p.q_stride + (long long)h * D;
      __nv_bfloat16* dst = p.q_out + t * p.q_out_stride + (long long)h * D;
      uint4 a = *reinterpret_cast<const uint4*>(src + ca * 8);
      uint4 b = *reinterpret_cast<const uint4*>(src + cb * 8);
      if (turn) {
        float cs[8], sn[8];
        load8(tab, cs);
        load8(tab + rd / 2, sn);
        if (p.interleaved) {
          rotate_neighbours(a, cs, sn);
          rotate_neighbours(b, cs + 4, sn + 4);
        } else {
          rotate_split(a, b, cs, sn);
        }
      }
      *reinterpret_cast<uint4*>(dst + ca * 8) = a;
      *reinterpret_cast<uint4*>(dst + cb * 8) = b;
      continue;
    }
    const int hk = h - Hq < p.Hkv ? h - Hq : h - Hq - p.Hkv;
    uint8_t* const blk =
        p.pages + kv4_block_at(page, p.Hkv, hk, p.page_shift, slot, Block::kBytes);
    if (h - Hq < p.Hkv) {
      const __nv_bfloat16* src = p.k + t * p.k_stride + (long long)hk * D;
      float a[8], b[8];
      widen8(*reinterpret_cast<const uint4*>(src + ca * 8), a);
      widen8(*reinterpret_cast<const uint4*>(src + cb * 8), b);
      if (turn) {
        float cs[8], sn[8];
        load8(tab, cs);
        load8(tab + rd / 2, sn);
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            turn_pair(a[2 * i], a[2 * i + 1], cs[i], sn[i]);
            turn_pair(b[2 * i], b[2 * i + 1], cs[4 + i], sn[4 + i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) turn_pair(a[i], b[i], cs[i], sn[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = __fmul_rn(a[i], p.k_inv);
        b[i] = __fmul_rn(b[i], p.k_inv);
      }
      // A group is two neighbouring chunks, whose threads tell each other
      // their largest magnitude: chunk c is thread c's first, thread c -
      // half's second, or (not turned) thread c / 2's.
      const float ta = top8(a), tb = top8(b);
      auto other = [&](int c) -> float {
        int from = c >> 1;
        bool second = (c & 1) != 0;
        if (!p.interleaved && c < 2 * half) {
          second = c >= half;
          from = second ? c - half : c;
        }
        const float x = __shfl_sync(group, ta, from, kPairs), y = __shfl_sync(group, tb, from, kPairs);
        return second ? y : x;
      };
      float sa, sb;
      const float ga = max_nan(ta, other(ca ^ 1)), gb = max_nan(tb, other(cb ^ 1));
      const uint32_t ba = kv4_scale(ga, sa), bb = kv4_scale(gb, sb);
      auto codes = [&](float (&y)[8], float top, float s) -> uint32_t {
        bound(y, top);
        const float inv = kv4_inverse(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = kv4_quotient(y[i], s, inv);
        return kv4_codes({y[0], y[2], y[4], y[6]}, {y[1], y[3], y[5], y[7]});
      };
      *reinterpret_cast<uint32_t*>(blk + Block::k_code(r) + ca * 4) = codes(a, ga, sa);
      *reinterpret_cast<uint32_t*>(blk + Block::k_code(r) + cb * 4) = codes(b, gb, sb);
      if ((ca & 1) == 0) blk[Block::k_scale(r) + (ca >> 1)] = (uint8_t)ba;
      if ((cb & 1) == 0) blk[Block::k_scale(r) + (cb >> 1)] = (uint8_t)bb;
    } else if (!before) {
      const __nv_bfloat16* src = p.v + t * p.v_stride + (long long)hk * D + pr * 16;
      // This row's group, and the next row's (else its own once more), divided by the
      // tensor's scale twice over, to spare registers.
      const uint4* const other_src = reinterpret_cast<const uint4*>(src + (after ? p.v_stride : 0));
      const uint4 mine[2] = {reinterpret_cast<const uint4*>(src)[0], reinterpret_cast<const uint4*>(src)[1]};
      const uint4 next[2] = {other_src[0], other_src[1]};
      const float tm = top16(mine, p.v_inv), tn = top16(next, p.v_inv);
      float sm, sn2;
      const uint32_t s_mine = kv4_scale(tm, sm), s_next = kv4_scale(tn, sn2);
      const float rm = kv4_inverse(sm), rn = kv4_inverse(sn2);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // Eight channels: an eighth of d = 64, half of one of d = 128.
        uint2* const dst = reinterpret_cast<uint2*>(
            blk + (D == 128 ? Block::v_code(r, pr) + 8 * i : Block::v_code(r, 2 * pr + i)));
        float e[8], o[8];
        quotients8(mine[i], p.v_inv, tm, sm, rm, e);
        quotients8(next[i], p.v_inv, tn, sn2, rn, o);
        uint2 x = make_uint2(kv4_codes({e[0], e[1], e[2], e[3]}, {o[0], o[1], o[2], o[3]}),
                             kv4_codes({e[4], e[5], e[6], e[7]}, {o[4], o[5], o[6], o[7]}));
        if (!after) {  // the other key's half stays
          const uint32_t keep = odd ? 0x0f0f0f0fu : 0xf0f0f0f0u;
          const uint2 old = *dst;
          x.x = x.x & ~keep | old.x & keep;
          x.y = x.y & ~keep | old.y & keep;
        }
        *dst = x;
      }
      uint8_t* const scale = blk + Block::v_scale(pr) + r;
      if (after)
        *reinterpret_cast<uint16_t*>(scale) = (uint16_t)(s_mine | s_next << 8);
      else
        *scale = (uint8_t)s_mine;
    }
  }
}

// A CTA takes `run` rows one after another: to find a row's place takes four rounds of
// loads of which each waits for the one before, to find the next one's none.
template <int D>
__global__ void __launch_bounds__(kThreads, 8) fa_kv4_append_kernel(const Kv4AppendParams p, int run) {
  launch_dependents();
  wait_prior_grid();
  RowPlace at = {-1, 0, 0, 0, -1};
  const int t0 = (int)blockIdx.x * run, t1 = min(t0 + run, p.T);
  for (int t = t0; t < t1; ++t) {
    at = place_row(p, t, at, p.rope_dim > 0 ? p.rope_len : -1);
    if (at.b >= 0) append_row<D>(p, t, at);
  }
  check_ranges(p);
}

// A thread takes 16 channels of a key or value head.
template <int D>
__device__ __forceinline__ void read_row(const Kv4ReadParams& p, int t, const RowPlace& at) {
  using Block = Kv4Block<D>;
  constexpr int kGroups = D / 16;
  const int page = at.page;
  const int slot = at.pos & (p.page_size - 1), r = slot & 15;
  for (int i = threadIdx.x; i < 2 * p.Hkv * kGroups; i += kThreads) {
    const int g = i % kGroups, hh = i / kGroups;
    const bool is_v = hh >= p.Hkv;
    const int h = is_v ? hh - p.Hkv : hh;
    const uint8_t* blk = p.pages + kv4_block_at(page, p.Hkv, h, p.page_shift, slot, Block::kBytes);
    uint32_t pair[8];  // channels 2i, 2i + 1 as fp16
    uint32_t sbyte;
    if (is_v) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint2 x = *reinterpret_cast<const uint2*>(
            blk + (D == 128 ? Block::v_code(r, g) + 8 * k : Block::v_code(r, 2 * g + k)));
        w[2 * k] = x.x;
        w[2 * k + 1] = x.y;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t both[4];
        e2m1_to_half(w[k], both);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          pair[2 * k + c] = __byte_perm(both[2 * c], both[2 * c + 1], (r & 1) ? 0x7632 : 0x5410);
      }
      sbyte = blk[Block::v_scale(g) + r];
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(blk + Block::k_code(r) + 8 * g);
      uint32_t a[4], b[4];
      e2m1_to_half(x.x, a);
      e2m1_to_half(x.y, b);
#pragma unroll
      for (int k = 0; k < 4; ++k) pair[k] = a[k], pair[4 + k] = b[k];
      sbyte = blk[Block::k_scale(r) + g];
    }
    const uint32_t s1 = e4m3_to_half(sbyte), s2 = __byte_perm(s1, s1, 0x1010);
    const float scale = is_v ? p.v_scale : p.k_scale;
    uint32_t out[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t x = half2_mul(pair[k], s2);  // exact
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
      out[k] = pack_bf16x2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
    }
    __nv_bfloat16* dst = (is_v ? p.v_out + t * p.v_out_stride : p.k_out + t * p.k_out_stride) +
                         (long long)h * D + g * 16;
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 8) fa_kv4_read_kernel(const Kv4ReadParams p, int run) {
  launch_dependents();
  wait_prior_grid();
  RowPlace at = {-1, 0, 0, 0, -1};
  const int t0 = (int)blockIdx.x * run, t1 = min(t0 + run, p.T);
  for (int t = t0; t < t1; ++t) {
    at = place_row(p, t, at, -1);
    if (at.b >= 0) read_row<D>(p, t, at);
  }
  check_ranges(p);
}

// Rows of a CTA: one as long as all CTAs run at once (8 an SM), then `most`.  (32 + 16
// heads, d = 128, in a graph: 256 single rows appended by one a CTA 5.1 us, by two 6.6;
// read back by one 2.7, by four 5.5; 1,216 single rows 7.5, 8.8 and 3.8, 6.3; 4 x 608
// rows 11.5, 10.6 and 5.2, 4.4; 16 x 1,024 rows 72, 69 and 26.5, 18.9.)
template <class Params>
int launch_rows(void (*kernel)(Params, int), const Params& p, int most, cudaStream_t stream) {
  const int run = p.T <= 1216 ? 1 : most;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(((long long)p.T + run - 1) / run), 1, 1);
  c.blockDim = dim3(kThreads, 1, 1);
  c.stream = stream;
  c.attrs = pdl;
  c.numAttrs = 1;
  if (cudaLaunchKernelEx(&c, kernel, p, run) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

}  // namespace

int launch_kv4_append(const Kv4AppendParams& p, int d, cudaStream_t stream) {
  return launch_rows(d == 128 ? fa_kv4_append_kernel<128> : fa_kv4_append_kernel<64>, p, 2, stream);
}
int launch_kv4_read(const Kv4ReadParams& p, int d, cudaStream_t stream) {
  return launch_rows(d == 128 ? fa_kv4_read_kernel<128> : fa_kv4_read_kernel<64>, p, 4, stream);
}

}  // namespace fa
