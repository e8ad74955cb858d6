// fa_paged4_prompt.cu -- the kernel for many query rows to a key/value head
// (fa_paged_prompt.cuh) over a cache held in 4 bits.
#include "fa_paged_launch.h"
#include "fa_paged_prompt.cuh"

namespace fa {
namespace {

template <int D, bool kNeg>
__global__ void __launch_bounds__(kPaged4Threads, 1)
    fa_paged4_prompt_kernel(const __grid_constant__ CUtensorMap tq,
                            const __grid_constant__ CUtensorMap to, const Paged4Params p,
                            const PagedPhase ph) {
  extern __shared__ uint8_t smem_raw[];
  prompt_cta<D, kNeg, false, true>(&tq, nullptr, nullptr, &to, p, ph, blockIdx.x, gridDim.x,
                                   smem_raw);
}

template <int D>
__global__ void __launch_bounds__(256, 3) fa_paged4_expand_kernel(const Paged4Params p, int n_min) {
  launch_dependents();
  wait_prior_grid();
  paged4_expand<D>(p, n_min, (int)(blockIdx.x * 8 + (threadIdx.x >> 5)), (int)gridDim.x * 8);
}

template <int D, bool kNeg>
int launch(const PagedMaps& t, const Paged4Params& p, const PagedPhase& ph,
           const cudaLaunchConfig_t& base) {
  cudaLaunchConfig_t c = base;
  c.blockDim = dim3(kPaged4Threads, 1, 1);
  c.dynamicSmemBytes = sizeof(PromptSmem<D>) + 1024;
  if (paged_kernel_ready<fa_paged4_prompt_kernel<D, kNeg>, kPaged4Regs>(c.dynamicSmemBytes) != FA_OK)
    return FA_ERR_LAUNCH;
  if (cudaLaunchKernelEx(&c, fa_paged4_prompt_kernel<D, kNeg>, t.q, t.o, p, ph) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

}  // namespace

int launch_paged4_prompt(const Paged4Params& p, PagedPhase& ph, int d,
                         const cudaLaunchConfig_t& base) {
  PagedMaps t;
  ph.tile_tokens = kTile / p.G;
  ph.unit_tokens = 2 * ph.tile_tokens;
  ph.slot_rows = kPairRows;
  ph.box_out = 32 % p.G == 0;
  int rc = make_tmap_rows(p.o, p.Hq, p.T, (long long)p.Hq * d, d, p.G, ph.box_out ? 32 / p.G : 1, &t.o);
  if (rc != FA_OK) return rc;
  rc = make_tmap_rows(p.q, p.Hq, p.T, p.q_stride, d, p.G, ph.tile_tokens, &t.q);
  if (rc != FA_OK) return rc;
  if (p.expand > 0) {
    cudaLaunchConfig_t c = base;
    c.gridDim = dim3((unsigned)p.ctas * 3, 1, 1);
    c.blockDim = dim3(256, 1, 1);
    const int n_min = kPaged4ExpandRows / p.G + 1;
    if (cudaLaunchKernelEx(&c, d == 128 ? fa_paged4_expand_kernel<128> : fa_paged4_expand_kernel<64>,
                           (const Paged4Params&)p, n_min) != cudaSuccess) {
      cudaGetLastError();
      return FA_ERR_LAUNCH;
    }
  }
  if (p.scale_log2 < 0.f) return d == 128 ? launch<128, true>(t, p, ph, base) : launch<64, true>(t, p, ph, base);
  return d == 128 ? launch<128, false>(t, p, ph, base) : launch<64, false>(t, p, ph, base);
}

}  // namespace fa
