// fa_kv.cu -- appending new keys and values to a paged cache, with the rotary
// position embedding of the new queries and keys applied on the way.
//
// A row t of the packed [T][heads][d] inputs belongs to the sequence b with
// cu_q[b] <= t < cu_q[b+1] and is its position
//     pos = seq_lens[b] - (cu_q[b+1] - t),
// the last new token being the sequence's last position.  Its key and value
// go to slot pos % page_size of page page_table[b][pos / page_size].  The
// rotation turns each pair (x, y) of the first rope_dim channels of a head by
// the angle whose cosine c and sine s the caller's table holds at pos:
//     x' = x c - y s,   y' = x s + y c,
// in fp32 from bf16 inputs, rounded to bf16 once.
//
// Bound by memory: q, k and v are read once and written once; the table rows
// (4 * rope_dim bytes) are shared by all heads of a row.  16,384 rows of 32
// query and 8 key/value heads, d = 128: 61 us, 6.7 TB/s of the 6.8 that a
// copy reaches; one row: 2.6 us, a launch and four rounds of loads of which each
// waits for the one before: the row ranges; the row's own and its length; the
// page number; the rotation table and the inputs.
#include <cuda_bf16.h>

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// (x, y) turned pairwise: eight pairs, x in one chunk and y in another.
__device__ __forceinline__ void rotate_split(uint4& x, uint4& y, const float* c, const float* s) {
  uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
  uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = bf2(xw[i]), b = bf2(yw[i]);
    const float c0 = c[2 * i], c1 = c[2 * i + 1], s0 = s[2 * i], s1 = s[2 * i + 1];
    xw[i] = pack_bf16x2(a.x * c0 - b.x * s0, a.y * c1 - b.y * s1);
    yw[i] = pack_bf16x2(a.x * s0 + b.x * c0, a.y * s1 + b.y * c1);
  }
}

// Neighbouring channels as pairs: four pairs of one chunk.
__device__ __forceinline__ void rotate_neighbours(uint4& x, const float* c, const float* s) {
  uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = bf2(xw[i]);
    xw[i] = pack_bf16x2(a.x * c[i] - a.y * s[i], a.x * s[i] + a.y * c[i]);
  }
}

__device__ __forceinline__ void load8(const float* src, float* dst) {
  const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
  dst[0] = a.x, dst[1] = a.y, dst[2] = a.z, dst[3] = a.w;
  dst[4] = b.x, dst[5] = b.y, dst[6] = b.z, dst[7] = b.w;
}

// One CTA per row.  A thread owns the same two 8-channel chunks of every
// kRows-th head: the chunks p and p + rope_dim/16 that hold a pair's two
// halves (or two neighbouring chunks), so that it reads its part of the table
// once.  The inputs are loaded last, when the row's place is known: a row of no
// sequence reads none.
constexpr int kAppendThreads = 128;

template <int D>
__device__ __forceinline__ void append_row(const KvAppendParams& p, int t) {
  constexpr int kPairs = D / 16;                   // chunk pairs of a head
  constexpr int kRows = kAppendThreads / kPairs;   // heads in one sweep of the CTA
  const int pr = threadIdx.x % kPairs, row = threadIdx.x / kPairs;
  const int rd = p.rope_dim;
  // The thread's chunks (8 channels each) and whether they are rotated.
  int ca = 2 * pr, cb = 2 * pr + 1;
  bool turn = false;
  if (p.interleaved) {
    turn = ca * 8 < rd;  // rope_dim is a multiple of 16: both chunks or neither
  } else if (pr < rd / 16) {
    ca = pr;
    cb = pr + rd / 16;
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
  const int slot = at.pos & (p.page_size - 1);
  const int Hq = p.q ? p.Hq : 0;
  for (int h = row; h < Hq + 2 * p.Hkv; h += kRows) {
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    bool rot = turn;
    if (h < Hq) {
      src = p.q + t * p.q_stride + (long long)h * D;
      dst = p.q_out + t * p.q_out_stride + (long long)h * D;
    } else {
      const int hk = (h - Hq) % p.Hkv;
      const bool is_v = h - Hq >= p.Hkv;
      src = (is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride) + (long long)hk * D;
      dst = (is_v ? p.v_pages : p.k_pages) +
            ((((long long)page * p.Hkv + hk) << p.page_shift) + slot) * D;
      rot = rot && !is_v;
    }
    uint4 a = *reinterpret_cast<const uint4*>(src + ca * 8);
    uint4 b = *reinterpret_cast<const uint4*>(src + cb * 8);
    if (rot) {
      if (p.interleaved) {
        rotate_neighbours(a, cs, sn);
        rotate_neighbours(b, cs + 4, sn + 4);
      } else {
        rotate_split(a, b, cs, sn);
      }
    }
    *reinterpret_cast<uint4*>(dst + ca * 8) = a;
    *reinterpret_cast<uint4*>(dst + cb * 8) = b;
  }
}

// The row's own sequence is looked at before anything is written; the ranges of
// all sequences, those without a row among them, by the CTAs' threads in turn.
// A thread's first is asked for at the start and looked at at the end, so that
// nothing waits for it (one row 2.55 us; asked for at the end 2.65, not looked at
// 2.45).  Twelve CTAs to an SM: 40 registers a thread (with 48, which the
// compiler would take, 16,384 rows take 61.2 us instead of 60.8).
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 12) fa_kv_append_kernel(const KvAppendParams p) {
  launch_dependents();
  wait_prior_grid();
  auto check = [&](int t0, int t1) {
    if (paged_range_ok(t0, t1, p.T)) return;
    int abort_flag = 0;
    report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedRows);
  };
  const long long first = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
  int t0 = 0, t1 = 0;
  if (first < p.B) {
    t0 = p.cu_q[first];
    t1 = p.cu_q[first + 1];
  }
  append_row<D>(p, (int)blockIdx.x);
  check(t0, t1);
  for (long long b = ((long long)blockIdx.x + p.T) * kAppendThreads + threadIdx.x; b < p.B;
       b += (long long)p.T * kAppendThreads)
    check(p.cu_q[b], p.cu_q[b + 1]);
}

}  // namespace

int launch_kv_append(const KvAppendParams& p, int d, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)p.T, 1, 1);
  c.blockDim = dim3(kAppendThreads, 1, 1);
  c.stream = stream;
  c.attrs = pdl;
  c.numAttrs = 1;
  const cudaError_t e = d == 128 ? cudaLaunchKernelEx(&c, fa_kv_append_kernel<128>, p)
                                 : cudaLaunchKernelEx(&c, fa_kv_append_kernel<64>, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

}  // namespace fa
