// fa_rope.cuh -- the rotary position embedding of 8-channel chunks of a row, as
// the appends to a paged cache apply it on the way.
#pragma once

#include "sm100_ptx.cuh"

namespace fa {

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

}  // namespace fa
