// Microscaled 4-bit values (OCP MXFP4): E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign),
// value 2 i in the low half of byte i, one UE8M0 scale byte per 32 consecutive values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

constexpr int kNanScale = 255;

// The scale byte of a block from its largest magnitude as bf16 bits: the smallest e + 127 with
// max <= 6 * 2^e.  6 = 1.5 * 2^2 and max = (1 + f / 128) 2^(E - 127), so e + 127 = E - 2, and one
// more where f > 64: a carry out of f + 63.  0 for what lies below 6 * 2^-127, 127 for a block of
// zeros, the NaN byte where a value is not finite (E2M1 has no code for it).
__device__ __forceinline__ int fp4_scale(uint32_t top) {
  if (top >= 0x7F80u) return kNanScale;
  const int s = (int)((top + 63) >> 7) - 2;
  return top == 0 ? 127 : (s < 0 ? 0 : s);
}

// 2^(byte - 127) for the conversions; byte 0 lies below the normal range.
__device__ __forceinline__ float scale_value(int byte) {
  return __uint_as_float(byte > 0 ? (uint32_t)byte << 23 : 0x00400000u);
}

// Eight bf16 values over the block's scale, rounded to nearest, ties to even (the hardware
// conversion: checked for every scale against the rounding written out).
__device__ __forceinline__ uint32_t pack_fp4x8(const uint4& v, int scale) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  if (scale == kNanScale) return 0;
  const float f = scale_value(scale);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v.x), f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v.y), f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v.z), f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v.w), f, 3);
  return w;
}

// The larger of two packed pairs of bf16 magnitudes, each half by itself.
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t pair_max8(const uint4& v) {
  constexpr uint32_t m = 0x7FFF7FFFu;
  return pair_max(pair_max(v.x & m, v.y & m), pair_max(v.z & m, v.w & m));
}

}  // namespace moe
