// fa_paged_launch.h -- what the two paged attention kernels' launchers share.
#pragma once

#include "fa_internal.h"
#include "fa_paged.cuh"

namespace fa {

// Tensor maps over q (a box per Q tile and 64 channels) and the pages.
struct PagedMaps {
  CUtensorMap q, k, v;
};

// The prompt kernel (fa_paged_prompt.cu): units of two 128-row Q tiles.
int launch_paged_prompt(const PagedMaps& t, const PagedParams& p, const PagedPhase& ph, int d,
                        const cudaLaunchConfig_t& base);

}  // namespace fa
