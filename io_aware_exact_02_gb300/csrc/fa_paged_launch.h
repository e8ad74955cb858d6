// fa_paged_launch.h -- what the two paged attention kernels' launchers share.
#pragma once

#include "fa_internal.h"
#include "fa_paged.cuh"

namespace fa {

// Tensor maps over q (a box per Q tile and 64 channels) and the pages.
struct PagedMaps {
  CUtensorMap q, k, v;
};

// Sets the kernel's shared memory on the current device and checks that it has
// the registers its warpgroups split.
template <class Kernel>
int paged_kernel_ready(Kernel* kernel, size_t smem) {
  cudaFuncAttributes attr;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess ||
      cudaFuncGetAttributes(&attr, kernel) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return attr.numRegs < kPagedRegs ? FA_ERR_LAUNCH : FA_OK;
}

// The prompt kernel (fa_paged_prompt.cu): units of two 128-row Q tiles.
int launch_paged_prompt(const PagedMaps& t, const PagedParams& p, const PagedPhase& ph, int d,
                        const cudaLaunchConfig_t& base);

}  // namespace fa
