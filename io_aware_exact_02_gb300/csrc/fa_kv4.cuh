// fa_kv4.cuh -- the 4-bit key/value cache: its layout, and numbers in and out.
//
// A group of 16 channels of a key (or value) row is held as 16 E2M1 codes
// (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) and one E4M3 scale s:
//     y = x / tensor scale,   s = E4M3(max |y| / 6),   code = E2M1(y / s),
//     value = code * s * tensor scale.
// A code has 2 significant bits and a scale 4, so code * s is exact in fp16 and
// in bf16, and the tensor's scale is left to the sums: scores times the keys',
// outputs times the values'.
//
// Blocks of 16 keys of one head, 18 d bytes:
//     K codes   [16 keys][d / 2]       a byte holds channels 2i (low) and 2i + 1
//     V codes   [2][8][4][d / 8]       half of 8 keys, eighth of the channels, key
//                                      pair, channel: a byte holds keys 2i (low), 2i + 1
//     K scales  [16 keys][d / 16]
//     V scales  [d / 16][16 keys]
// Each operand of the tensor core's m16n8k16 product is then read from a block
// by the lanes that need it as whole 16-byte (d = 64: 8-byte) pieces of
// consecutive addresses, its pairs of neighbours (channels of a key; keys of a
// value channel) in one byte, which one conversion turns into a register.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace fa {

// Offsets in a block.
template <int D>
struct Kv4Block {
  static constexpr int kBytes = 18 * D;
  static constexpr int kEighth = D / 8;  // channels
  static __host__ __device__ constexpr int k_code(int r) { return r * (D / 2); }
  // Channel eighth * kEighth of key r: the byte that its pair of keys shares.
  static __host__ __device__ constexpr int v_code(int r, int eighth) {
    return 8 * D + (((r >> 3) * 8 + eighth) * 4 + ((r & 7) >> 1)) * kEighth;
  }
  static __host__ __device__ constexpr int k_scale(int r) { return 16 * D + r * (D / 16); }
  static __host__ __device__ constexpr int v_scale(int group) { return 17 * D + group * 16; }
};

// Byte offset of the block of a page's slot: 32-bit factors (num_pages * Hkv is below
// 2^31, a page's blocks of a head below 2^16 bytes), a 64-bit product.
__device__ __forceinline__ long long kv4_block_at(int page, int Hkv, int h, int page_shift, int slot,
                                                  int block_bytes) {
  return (long long)((unsigned long long)(uint32_t)(page * Hkv + h) *
                     (uint32_t)(block_bytes << (page_shift - 4))) +
         (slot >> 4) * block_bytes;
}

// Four bytes of two codes each to pairs of fp16, exactly.
__device__ __forceinline__ void e2m1_to_half(uint32_t bytes, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(bytes));
}
// Two E4M3 numbers to a pair of fp16, exactly.
__device__ __forceinline__ uint32_t e4m3_to_half(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The larger of two numbers, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The scale of a group whose largest magnitude is top, as a byte and a number.
// Above 6 * 448 (and for infinities) it is 448, for NaN it is NaN.
__device__ __forceinline__ uint32_t kv4_scale(float top, float& s) {
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(__fdiv_rn(top, 6.f)));
  s = __half2float(__ushort_as_half((unsigned short)(e4m3_to_half(two) & 0xffffu)));
  return two & 0xffu;
}
// The inverse of a scale, for kv4_quotient: 0 for a scale of 0, whose codes are 0.
__device__ __forceinline__ float kv4_inverse(float s) { return s == 0.f ? 0.f : __frcp_rn(s); }
// y / s rounded to nearest, of a y that is finite: a product with the rounded inverse
// r, and what that leaves over once more (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990: so corrected, a quotient
// within one unit of the last place is the rounded one).  A true quotient halfway
// between two codes is then met exactly.
__device__ __forceinline__ float kv4_quotient(float y, float s, float r) {
  const float q = __fmul_rn(y, r);
  return __fmaf_rn(__fmaf_rn(-q, s, y), r, q);
}
// Eight quotients to codes, number 2i in the lower half of byte i and 2i + 1 in the
// upper one; halfway cases to the even code, beyond the range to 6.
__device__ __forceinline__ uint32_t kv4_codes(const float (&lo)[4], const float (&hi)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %5, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %6, %2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %7, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %4;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(lo[0]), "f"(lo[1]), "f"(lo[2]), "f"(lo[3]), "f"(hi[0]), "f"(hi[1]), "f"(hi[2]), "f"(hi[3]));
  return r;
}

// The power of two that takes a query row, whose largest magnitude has the bits
// `top` of an fp32 number, to [2^14, 2^15), where fp16 holds every channel of at
// least 2^-31 of that one, and the others to 2^-39 of it; as an exponent.  At most
// 126, whose inverse is a normal number too: it makes every bf16 number a multiple of
// 2^-7, so rows that it leaves below 2^14 are held whole.  Zeros, infinities and NaN
// stay.
__device__ __forceinline__ int kv4_row_exponent(uint32_t top) {
  return top > 0u && top < 0x7f800000u ? min(14 - ((int)(top >> 23) - 127), 126) : 0;
}
__device__ __forceinline__ float kv4_pow2(int e) { return __int_as_float((e + 127) << 23); }
// The larger of `top` and the magnitudes of a pair of bf16 numbers, as bits of
// fp32 numbers (which compare as integers).
__device__ __forceinline__ uint32_t kv4_top(uint32_t top, uint32_t pair) {
  return max(top, max(pair << 16 & 0x7fffffffu, pair & 0x7fff0000u));
}

}  // namespace fa
