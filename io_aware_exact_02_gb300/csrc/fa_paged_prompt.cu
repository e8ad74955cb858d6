// fa_paged_prompt.cu -- the kernel for many query rows to a key/value head
// (fa_paged_prompt.cuh) on all CTAs.
#include "fa_paged_launch.h"
#include "fa_paged_prompt.cuh"

namespace fa {
namespace {

template <int D, bool kNeg>
__global__ void __launch_bounds__(kPagedThreads, 1)
    fa_paged_prompt_kernel(const __grid_constant__ CUtensorMap tq,
                           const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv,
                           const __grid_constant__ CUtensorMap to, const PagedParams p,
                           const PagedPhase ph) {
  extern __shared__ uint8_t smem_raw[];
  prompt_cta<D, kNeg, false>(&tq, &tk, &tv, &to, p, ph, blockIdx.x, gridDim.x, smem_raw);
}

template <int D, bool kNeg>
int launch_prompt(const PagedMaps& t, const PagedParams& p, const PagedPhase& ph,
                  const cudaLaunchConfig_t& base) {
  static_assert(sizeof(PromptSmem<D>) + 1024 <= 232448,
                "prompt shared memory above the 227 KB a CTA may have");
  cudaLaunchConfig_t c = base;
  c.blockDim = dim3(kPagedThreads, 1, 1);
  c.dynamicSmemBytes = sizeof(PromptSmem<D>) + 1024;
  if (paged_kernel_ready<fa_paged_prompt_kernel<D, kNeg>>(c.dynamicSmemBytes) != FA_OK)
    return FA_ERR_LAUNCH;
  if (cudaLaunchKernelEx(&c, fa_paged_prompt_kernel<D, kNeg>, t.q, t.k, t.v, t.o, p,
                         ph) !=
          cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

}  // namespace

int launch_paged_prompt(const PagedMaps& t, const PagedParams& params, const PagedPhase& ph, int d,
                        const cudaLaunchConfig_t& base) {
  PagedParams p = params;
  // A zero scale makes every visible key equal; it runs as the smallest normal
  // positive scale, whose exponents round to exactly 0.
  if (p.scale_log2 == 0.f) p.scale_log2 = 1.17549435e-38f;
  if (p.scale_log2 < 0.f)
    return d == 128 ? launch_prompt<128, true>(t, p, ph, base)
                    : launch_prompt<64, true>(t, p, ph, base);
  return d == 128 ? launch_prompt<128, false>(t, p, ph, base)
                  : launch_prompt<64, false>(t, p, ph, base);
}

}  // namespace fa
