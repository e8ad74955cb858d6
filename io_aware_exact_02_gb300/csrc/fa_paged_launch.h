// fa_paged_launch.h -- what the two paged attention kernels' launchers share.
#pragma once

#include <atomic>

#include "fa_internal.h"
#include "fa_paged.cuh"

namespace fa {

// Tensor maps over q (a box per Q tile and 64 channels), the pages, and o (a
// box per 32 rows and 64 channels, where a phase stores such: box_out).
struct PagedMaps {
  CUtensorMap q, k, v, o;
};

// Sets the kernel's shared memory on the current device and checks that it has
// the registers its warpgroups split, once per device.
template <auto* kernel>
int paged_kernel_ready(size_t smem) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  static std::atomic<unsigned long long> ready{0};  // one per kernel, a bit per device
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (ready.load(std::memory_order_relaxed) & bit) return FA_OK;
  cudaFuncAttributes attr;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess ||
      cudaFuncGetAttributes(&attr, kernel) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  if (attr.numRegs < kPagedRegs) return FA_ERR_LAUNCH;
  ready.fetch_or(bit, std::memory_order_relaxed);
  return FA_OK;
}

// The prompt kernel (fa_paged_prompt.cu): units of two 128-row Q tiles.
int launch_paged_prompt(const PagedMaps& t, const PagedParams& p, const PagedPhase& ph, int d,
                        const cudaLaunchConfig_t& base);

// Both kernels side by side (fa_paged_duo.cu): phase pa's units of 256 rows
// (Q map t.q) and phase pb's of 8 or 16 (tq_b).
int launch_paged_duo(const PagedMaps& t, const CUtensorMap& tq_b, const PagedParams& p,
                     const PagedPhase& pa, const PagedPhase& pb, int d,
                     const cudaLaunchConfig_t& base);

}  // namespace fa
