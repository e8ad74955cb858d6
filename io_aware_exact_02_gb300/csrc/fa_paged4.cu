// fa_paged4.cu -- attention over a paged key/value cache held in 4 bits.
//
// One warp per query row and head, with the online softmax over 32 keys at a
// time: a lane takes the scores of one key, then its share of the channels of
// the 32 values.
#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_paged.cuh"
#include "fa_paged4_decode.cuh"
#include "fa_paged_launch.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) fa_paged4_rows_kernel(const Paged4Params p, int n_min) {
  using Block = Kv4Block<D>;
  constexpr int kPer = D / 32;
  __shared__ float qs[kWarps][D];
  launch_dependents();
  wait_prior_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = (int)blockIdx.x, hq = (int)blockIdx.y * kWarps + warp;
  if (blockIdx.y == 0)
    for (long long b = (long long)t * blockDim.x + threadIdx.x; b < p.B; b += (long long)p.T * blockDim.x) {
      int abort_flag = 0;
      if (!paged_range_ok(p.cu_q[b], p.cu_q[b + 1], p.T))
        report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedRows);
    }
  const PagedRow at = paged_row(p.cu_q, p.seq_lens, p.B, p.T, t, p.status);
  if (at.b < 0 || hq >= p.Hq || p.cu_q[at.b + 1] - p.cu_q[at.b] < n_min) return;
  int abort_flag = 0;
  int len = p.seq_lens[at.b];
  const int cap = p.max_pages << p.page_shift;
  if (len < 0 || len > cap) {
    if (lane == 0) report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedLength);
    return;
  }
  const int lim = p.causal ? max(0, min(at.pos + 1, len)) : len;
  const int hk = hq / p.G;
  float* q = qs[warp];
  for (int i = lane; i < D; i += 32)
    q[i] = __bfloat162float(p.q[t * p.q_stride + (long long)hq * D + i]);
  __syncwarp();
  const float c2 = p.scale_log2 * p.k_scale, ninf = __int_as_float(0xff800000);
  float m = ninf, l = 0.f, acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  for (int k0 = 0; k0 < lim; k0 += 32) {
    const int key = k0 + lane;
    const uint8_t* blk = nullptr;
    if (key < lim) {
      const int page = p.page_table[(long long)at.b * p.max_pages + (key >> p.page_shift)];
      if (page < 0 || page >= p.num_pages)
        report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPage);
      else
        blk = p.pages + kv4_block_at(page, p.Hkv, hk, p.page_shift, key & (p.page_size - 1), Block::kBytes);
    }
    float s = ninf;
    if (blk != nullptr) {
      s = 0.f;
      const int r = key & 15;
      for (int g = 0; g < D / 16; ++g) {
        const uint2 x = *reinterpret_cast<const uint2*>(blk + Block::k_code(r) + 8 * g);
        uint32_t w[8];
        e2m1_to_half(x.x, reinterpret_cast<uint32_t(&)[4]>(w[0]));
        e2m1_to_half(x.y, reinterpret_cast<uint32_t(&)[4]>(w[4]));
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          part += f.x * q[16 * g + 2 * i] + f.y * q[16 * g + 2 * i + 1];
        }
        const uint32_t sc = e4m3_to_half(blk[Block::k_scale(r) + g]);
        s += part * __half2float(__ushort_as_half((unsigned short)(sc & 0xffffu)));
      }
      s *= c2;
    }
    float top = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, m);
    const bool none = __all_sync(0xffffffffu, s == ninf);
    if (none) continue;
    const float old = m == ninf ? 0.f : exp2f(m - top), e = exp2f(s - top);
    m = top;
    l = l * old + e;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] *= old;
    for (int k = 0; k < 32; ++k) {
      const uint8_t* vb = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(blk), k));
      const float pk = __shfl_sync(0xffffffffu, e, k);
      if (vb == nullptr || pk == 0.f) continue;
      const int r = (k0 + k) & 15;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int c = lane * kPer + i;
        uint32_t w[4];
        e2m1_to_half(vb[Block::v_code(r, c / Block::kEighth) + c % Block::kEighth], w);
        const uint32_t sc = e4m3_to_half(vb[Block::v_scale(c / 16) + r]);
        const float v = __half2float(__ushort_as_half((unsigned short)((r & 1) ? w[0] >> 16 : w[0] & 0xffffu)));
        acc[i] += pk * (v * __half2float(__ushort_as_half((unsigned short)(sc & 0xffffu))));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const long long row = (long long)t * p.Hq + hq;
  const float inv = l == 0.f ? 0.f : p.v_scale / l;
#pragma unroll
  for (int i = 0; i < kPer; ++i) p.o[row * D + lane * kPer + i] = __float2bfloat16(acc[i] * inv);
  if (lane == 0) p.lse[row] = l == 0.f ? ninf : (m + log2f(l)) * kLn2;
}

template <int D, int R>
__global__ void __launch_bounds__(Decode4Cfg<D, R>::kThreads, Decode4Cfg<D, R>::kCtas)
    fa_paged4_decode_kernel(const Paged4Params p, const PagedPhase ph, int subs) {
  extern __shared__ uint8_t smem_raw[];
  decode4_cta<D, R>(p, ph, subs, blockIdx.x, gridDim.x, smem_raw);
}

template <int D, int R>
int launch_decode(const Paged4Params& p, const PagedPhase& ph, int subs,
                  const cudaLaunchConfig_t& base) {
  static_assert((sizeof(Decode4Smem<D, R>) + 128 + 1024) * Decode4Cfg<D, R>::kCtas <= 233472,
                "shared memory above the 228 KB of an SM, of which a CTA takes 1 KB more");
  cudaLaunchConfig_t c = base;
  c.blockDim = dim3(Decode4Cfg<D, R>::kThreads, 1, 1);
  c.dynamicSmemBytes = sizeof(Decode4Smem<D, R>) + 128;
  if (paged_kernel_ready<fa_paged4_decode_kernel<D, R>, 0>(c.dynamicSmemBytes) != FA_OK)
    return FA_ERR_LAUNCH;
  if (cudaLaunchKernelEx(&c, fa_paged4_decode_kernel<D, R>, p, ph, subs) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

template <int D>
int launch_paged4_d(const Paged4Params& p, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.stream = stream;
  c.attrs = pdl;
  c.numAttrs = 1;
  const Paged4Form f = paged4_form(p.T, p.B, p.G, p.max_q);
  const Paged4Workspace w = paged4_workspace_layout(D, f);
  auto at = [&](size_t offset) { return reinterpret_cast<float*>(p.workspace + offset); };
  int rc;
  if (f.prompt) {
    c.gridDim = dim3((unsigned)p.T, (unsigned)((p.Hq + kWarps - 1) / kWarps), 1);
    c.blockDim = dim3(32 * kWarps, 1, 1);
    if (cudaLaunchKernelEx(&c, fa_paged4_rows_kernel<D>, p, f.small_tokens + 1) != cudaSuccess) {
      cudaGetLastError();
      return FA_ERR_LAUNCH;
    }
  }
  c.gridDim = dim3((unsigned)p.ctas, 1, 1);
  if (f.rows > 0) {
    Paged4Params q = p;  // its heads are runs of a token's
    q.G = f.heads;
    q.Hkv = p.Hkv * f.subs;
    q.ctas = p.ctas * kPaged4CtasPerSm;
    c.gridDim.x = (unsigned)q.ctas;
    PagedPhase ph = {};
    ph.rec = p.workspace + w.rec[0];
    ph.slot_o = at(w.slot_o[0]);
    ph.slot_lse = at(w.slot_lse[0]);
    ph.n_max = f.prompt ? f.small_tokens : 0x7fffffff;
    ph.unit_tokens = ph.tile_tokens = f.rows / f.heads;
    ph.slot_rows = f.rows;
    rc = f.rows == 8 ? launch_decode<D, 8>(q, ph, f.subs, c) : launch_decode<D, 16>(q, ph, f.subs, c);
    if (rc != FA_OK) return rc;
    if ((rc = launch_paged_merge(q, ph, D, 4, c)) != FA_OK) return rc;
  }
  return FA_OK;
}

}  // namespace

int launch_fwd_paged4(const Paged4Params& p, int d, cudaStream_t stream) {
  return d == 128 ? launch_paged4_d<128>(p, stream) : launch_paged4_d<64>(p, stream);
}

}  // namespace fa
