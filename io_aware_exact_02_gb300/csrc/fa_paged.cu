// fa_paged.cu -- attention over a paged key/value cache.
#include "fa_internal.h"
#include "fa_paged.cuh"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;

// One warp per (row, query head): lane l holds channels l*D/32 .. of q and of
// the O accumulator and walks the keys one at a time with the running maximum
// and sum of the softmax.
template <int D>
__global__ void __launch_bounds__(128) fa_paged_simple_kernel(const PagedParams p) {
  wait_prior_grid();
  constexpr int kPer = D / 32;
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= (long long)p.T * p.Hq) return;
  const int t = (int)(w / p.Hq), h = (int)(w % p.Hq), hk = h / p.G;
  const PagedRow at = paged_row(p.cu_q, p.seq_lens, p.B, p.T, t, p.status);
  if (at.b < 0) return;
  const long long cap = (long long)p.max_pages << p.page_shift;
  int abort_flag = 0;
  long long len = p.seq_lens[at.b];
  if (len < 0 || len > cap) {
    if (lane == 0) report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedLength);
    len = len < 0 ? 0 : cap;
  }
  long long lim = p.causal ? min((long long)at.pos + 1, len) : len;
  float q[kPer], o[kPer];
  for (int i = 0; i < kPer; ++i) {
    q[i] = __bfloat162float(p.q[t * p.q_stride + (long long)h * D + lane * kPer + i]) * p.scale_log2;
    o[i] = 0.f;
  }
  const float ninf = __int_as_float(0xff800000);
  float m = ninf, l = 0.f;
  for (int j = 0; j < lim; ++j) {
    const int pi = j >> p.page_shift;
    const int page = j < p.prefix_len ? p.prefix_pages[pi]
                                      : p.page_table[(long long)at.b * p.max_pages + pi];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) report_status(p.status, &abort_flag, FA_ERR_PAGE, kSitePagedPage);
      continue;
    }
    const long long off = ((((long long)page * p.Hkv + hk) << p.page_shift) + (j & (p.page_size - 1))) * D;
    float s = 0.f;
    for (int i = 0; i < kPer; ++i) s += q[i] * __bfloat162float(p.k_pages[off + lane * kPer + i]);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s), base = mn == ninf ? 0.f : mn;
    const float a = exp2f(m - base), e = exp2f(s - base);
    l = l * a + e;
    for (int i = 0; i < kPer; ++i)
      o[i] = o[i] * a + e * __bfloat162float(p.v_pages[off + lane * kPer + i]);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int i = 0; i < kPer; ++i)
    p.o[((long long)t * p.Hq + h) * D + lane * kPer + i] = __float2bfloat16(o[i] * inv);
  if (lane == 0) p.lse[(long long)t * p.Hq + h] = l > 0.f ? (m + log2f(l)) * kLn2 : ninf;
}

}  // namespace

int launch_fwd_paged(const PagedParams& p, int d, cudaStream_t stream) {
  const long long warps = (long long)p.T * p.Hq;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)((warps + 3) / 4), 1, 1);
  c.blockDim = dim3(128, 1, 1);
  c.stream = stream;
  c.attrs = pdl;
  c.numAttrs = 1;
  const cudaError_t e = d == 128 ? cudaLaunchKernelEx(&c, fa_paged_simple_kernel<128>, p)
                                 : cudaLaunchKernelEx(&c, fa_paged_simple_kernel<64>, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

}  // namespace fa
