// fa_paged4_prompt.cu -- the kernel for many query rows to a key/value head
// (fa_paged_prompt.cuh) over a cache held in 4 bits, and the one that makes the fp16
// tiles of long prompts before it (24 warps an SM, a quarter of a K or V tile each: 15 us
// for 67 MB; 12 warps, a quarter of both each, 17; stored by each lane itself 26).
#include "fa_paged_launch.h"
#include "fa_paged_prompt.cuh"

namespace fa {
namespace {

constexpr int kExpandWarps = 4;

template <bool kWhole>
constexpr int kPromptThreads = kWhole ? kPagedThreads : kPaged4Threads;

template <int D, bool kNeg, bool kWhole>
__global__ void __launch_bounds__(kPromptThreads<kWhole>, 1)
    fa_paged4_prompt_kernel(const __grid_constant__ CUtensorMap tq,
                            const __grid_constant__ CUtensorMap to, const Paged4Params p,
                            const PagedPhase ph) {
  extern __shared__ uint8_t smem_raw[];
  prompt_cta<D, kNeg, false, true, kWhole>(&tq, nullptr, nullptr, &to, p, ph, blockIdx.x, gridDim.x,
                                           smem_raw);
}

template <int D>
struct alignas(128) ExpandSmem {
  uint8_t stage[kExpandWarps][32 * D * 2];
};

template <int D>
__global__ void __launch_bounds__(32 * kExpandWarps, 6)
    fa_paged4_expand_kernel(const Paged4Params p, int n_min) {
  extern __shared__ uint8_t smem_raw[];
  ExpandSmem<D>& sm = *reinterpret_cast<ExpandSmem<D>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  launch_dependents();
  wait_prior_grid();
  const int warp = threadIdx.x >> 5;
  paged4_expand<D>(p, n_min, (int)blockIdx.x * kExpandWarps + warp, (int)gridDim.x * kExpandWarps,
                   sm.stage[warp]);
}

template <int D>
int launch_expand(const Paged4Params& p, const cudaLaunchConfig_t& base) {
  cudaLaunchConfig_t c = base;
  c.gridDim = dim3((unsigned)p.ctas * 6, 1, 1);
  c.blockDim = dim3(32 * kExpandWarps, 1, 1);
  c.dynamicSmemBytes = sizeof(ExpandSmem<D>) + 128;
  if (paged_kernel_ready<fa_paged4_expand_kernel<D>, 0>(c.dynamicSmemBytes) != FA_OK)
    return FA_ERR_LAUNCH;
  if (cudaLaunchKernelEx(&c, fa_paged4_expand_kernel<D>, p, p.expand_n_min) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

template <int D, bool kNeg, bool kWhole>
int launch(const PagedMaps& t, const Paged4Params& p, const PagedPhase& ph,
           const cudaLaunchConfig_t& base) {
  cudaLaunchConfig_t c = base;
  c.blockDim = dim3(kPromptThreads<kWhole>, 1, 1);
  c.dynamicSmemBytes = sizeof(PromptSmem<D>) + 1024;
  constexpr int kRegs = kWhole ? kPagedRegs : kPaged4Regs;
  if (paged_kernel_ready<fa_paged4_prompt_kernel<D, kNeg, kWhole>, kRegs>(c.dynamicSmemBytes) != FA_OK)
    return FA_ERR_LAUNCH;
  if (cudaLaunchKernelEx(&c, fa_paged4_prompt_kernel<D, kNeg, kWhole>, t.q, t.o, p, ph) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

template <bool kWhole>
int launch_whole(const PagedMaps& t, const Paged4Params& p, const PagedPhase& ph, int d,
                 const cudaLaunchConfig_t& base) {
  if (p.scale_log2 < 0.f)
    return d == 128 ? launch<128, true, kWhole>(t, p, ph, base) : launch<64, true, kWhole>(t, p, ph, base);
  return d == 128 ? launch<128, false, kWhole>(t, p, ph, base) : launch<64, false, kWhole>(t, p, ph, base);
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
    rc = d == 128 ? launch_expand<128>(p, base) : launch_expand<64>(p, base);
    if (rc != FA_OK) return rc;
  }
  if (p.whole) return launch_whole<true>(t, p, ph, d, base);
  return launch_whole<false>(t, p, ph, d, base);
}

}  // namespace fa
