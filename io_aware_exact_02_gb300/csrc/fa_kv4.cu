// fa_kv4.cu -- appending new keys and values to a paged cache held in 4 bits,
// with the rotary position embedding of the new queries and keys applied on the
// way, and reading rows of it back.
//
// Rows, positions and the rotation are those of fa_kv.cu; the numbers and their
// layout those of fa_kv4.cuh.  The rotated keys are quantised from fp32, each
// product and difference of the rotation rounded by itself, so that a code does
// not depend on how the compiler joins them.
//
// A byte of V holds a pair of neighbouring keys.  The row of the even slot
// writes both where the odd slot's row is new too; an odd slot whose neighbour
// was there before keeps that one's half.
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

// A value row's 16 channels of one group, divided by the tensor's scale.
__device__ __forceinline__ void quantize_group(const __nv_bfloat16* src, float inv, uint32_t (&code)[2],
                                               uint32_t& scale) {
  float y[16], s;
  widen8(reinterpret_cast<const uint4*>(src)[0], y);
  widen8(reinterpret_cast<const uint4*>(src)[1], y + 8);
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(y[i], inv);
  scale = kv4_scale(max_nan(top8(y), top8(y + 8)), s);
  code[0] = kv4_codes(y, s);
  code[1] = kv4_codes(y + 8, s);
}

// Eight codes of the even key and eight of the odd one to eight bytes.
__device__ __forceinline__ uint2 join_codes(uint32_t even, uint32_t odd) {
  uint32_t r[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    r[h] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = (even >> (16 * h + 4 * i)) & 15u, hi = (odd >> (16 * h + 4 * i)) & 15u;
      r[h] |= (lo | hi << 4) << (8 * i);
    }
  }
  return make_uint2(r[0], r[1]);
}

// One CTA per row, threads as in fa_kv.cu: a thread owns two 8-channel chunks of
// every kRows-th head.
template <int D>
__device__ __forceinline__ void append_row(const Kv4AppendParams& p, int t) {
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
  const PagedRow at = paged_row(p.cu_q, p.seq_lens, p.B, p.T, t, p.status);
  if (at.b < 0) return;
  const long long cap = (long long)p.max_pages << p.page_shift;
  int abort_flag = 0;
  if (at.pos < 0 || at.pos >= cap || (rd > 0 && at.pos >= p.rope_len)) {
    if (threadIdx.x == 0) report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPosition);
    return;
  }
  const int page = p.page_table[(long long)at.b * p.max_pages + (at.pos >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPage);
    return;
  }
  float cs[8], sn[8];
  if (turn) {
    const float* tab = p.rope + (long long)at.pos * rd;
    load8(tab + pr * 8, cs);
    load8(tab + rd / 2 + pr * 8, sn);
  }
  const int slot = at.pos & (p.page_size - 1), r = slot & 15;
  const int Hq = p.q ? p.Hq : 0;
  const bool odd = (r & 1) != 0;
  const bool before = odd && t > p.cu_q[at.b], after = !odd && t + 1 < p.cu_q[at.b + 1];
  const unsigned group = (kPairs == 8 ? 0xffu : 0xfu) << ((threadIdx.x & 31) & ~(kPairs - 1));
  for (int h = row; h < Hq + 2 * p.Hkv; h += kRows) {
    if (h < Hq) {
      const __nv_bfloat16* src = p.q + t * p.q_stride + (long long)h * D;
      __nv_bfloat16* dst = p.q_out + t * p.q_out_stride + (long long)h * D;
      uint4 a = *reinterpret_cast<const uint4*>(src + ca * 8);
      uint4 b = *reinterpret_cast<const uint4*>(src + cb * 8);
      if (turn) {
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
      const uint32_t ba = kv4_scale(max_nan(ta, other(ca ^ 1)), sa);
      const uint32_t bb = kv4_scale(max_nan(tb, other(cb ^ 1)), sb);
      *reinterpret_cast<uint32_t*>(blk + Block::k_code(r) + ca * 4) = kv4_codes(a, sa);
      *reinterpret_cast<uint32_t*>(blk + Block::k_code(r) + cb * 4) = kv4_codes(b, sb);
      if ((ca & 1) == 0) blk[Block::k_scale(r) + (ca >> 1)] = (uint8_t)ba;
      if ((cb & 1) == 0) blk[Block::k_scale(r) + (cb >> 1)] = (uint8_t)bb;
    } else if (!before) {
      const __nv_bfloat16* src = p.v + t * p.v_stride + (long long)hk * D + pr * 16;
      uint32_t mine[2], next[2] = {0u, 0u}, s_mine, s_next = 0;
      quantize_group(src, p.v_inv, mine, s_mine);
      if (after) quantize_group(src + p.v_stride, p.v_inv, next, s_next);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // Eight channels: an eighth of d = 64, half of one of d = 128.
        uint2* const dst = reinterpret_cast<uint2*>(
            blk + (D == 128 ? Block::v_code(r, pr) + 8 * i : Block::v_code(r, 2 * pr + i)));
        uint2 x;
        if (odd) {
          const uint2 old = *dst;
          x = join_codes(0u, mine[i]);
          x.x |= old.x & 0x0f0f0f0fu;
          x.y |= old.y & 0x0f0f0f0fu;
        } else {
          x = join_codes(mine[i], next[i]);
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

template <int D>
__global__ void __launch_bounds__(kThreads) fa_kv4_append_kernel(const Kv4AppendParams p) {
  launch_dependents();
  wait_prior_grid();
  append_row<D>(p, (int)blockIdx.x);
  // The ranges of all sequences, those without a row among them.
  for (long long b = (long long)blockIdx.x * kThreads + threadIdx.x; b < p.B;
       b += (long long)p.T * kThreads) {
    int abort_flag = 0;
    if (!paged_range_ok(p.cu_q[b], p.cu_q[b + 1], p.T))
      report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedRows);
  }
}

// One CTA per row; a thread takes 16 channels of a key or value head.
template <int D>
__global__ void __launch_bounds__(kThreads) fa_kv4_read_kernel(const Kv4ReadParams p) {
  using Block = Kv4Block<D>;
  constexpr int kGroups = D / 16;
  launch_dependents();
  wait_prior_grid();
  const int t = (int)blockIdx.x;
  for (long long b = (long long)t * kThreads + threadIdx.x; b < p.B; b += (long long)p.T * kThreads) {
    int abort_flag = 0;
    if (!paged_range_ok(p.cu_q[b], p.cu_q[b + 1], p.T))
      report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedRows);
  }
  const PagedRow at = paged_row(p.cu_q, p.seq_lens, p.B, p.T, t, p.status);
  if (at.b < 0) return;
  int abort_flag = 0;
  if (at.pos < 0 || at.pos >= (long long)p.max_pages << p.page_shift) {
    if (threadIdx.x == 0) report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPosition);
    return;
  }
  const int page = p.page_table[(long long)at.b * p.max_pages + (at.pos >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPage);
    return;
  }
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

template <class Params>
int launch_rows(void (*kernel)(Params), const Params& p, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)p.T, 1, 1);
  c.blockDim = dim3(kThreads, 1, 1);
  c.stream = stream;
  c.attrs = pdl;
  c.numAttrs = 1;
  if (cudaLaunchKernelEx(&c, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

}  // namespace

int launch_kv4_append(const Kv4AppendParams& p, int d, cudaStream_t stream) {
  return launch_rows(d == 128 ? fa_kv4_append_kernel<128> : fa_kv4_append_kernel<64>, p, stream);
}
int launch_kv4_read(const Kv4ReadParams& p, int d, cudaStream_t stream) {
  return launch_rows(d == 128 ? fa_kv4_read_kernel<128> : fa_kv4_read_kernel<64>, p, stream);
}

}  // namespace fa
