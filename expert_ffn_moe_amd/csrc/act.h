// Activations of the grouped linear products, their derivatives and the 8-bit form in which
// the pre-activations are kept for the backward pass.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.h"
#include "../../include/moe.h"

namespace moe {

// The hardware reciprocal (1 ulp) in place of the exact division's ten instructions; results
// below the normal range are zero.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// gelu in its tanh form, 0.5 z (1 + tanh u) = z sigma(2 u) with u = r (z + c z^3).
constexpr float kGeluR2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {  // wave-uniform
    case MOE_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case MOE_ACT_RELU2: return z < 0.0f ? 0.0f : z * z;
    case MOE_ACT_SILU: return z * sigmoid(z);
    case MOE_ACT_GELU_TANH: return z * sigmoid(kGeluR2 * (z + kGeluC * z * z * z));
    default: return z;
  }
}

// act(z) and act'(z).  The gelu's second term is dropped where sigma (1 - sigma) is zero:
// there z^2 may overflow, and the product's limit is zero.
__device__ __forceinline__ void act_both(int act, float z, float& f, float& df) {
  switch (act) {  // wave-uniform
    case MOE_ACT_RELU:
      f = z < 0.0f ? 0.0f : z;
      df = z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);  // NaN stays NaN
      return;
    case MOE_ACT_RELU2:
      f = z < 0.0f ? 0.0f : z * z;
      df = z < 0.0f ? 0.0f : 2.0f * z;
      return;
    case MOE_ACT_SILU: {
      const float s = sigmoid(z);
      f = z * s;
      df = s * (1.0f + z * (1.0f - s));
      return;
    }
    case MOE_ACT_GELU_TANH: {
      const float s = sigmoid(kGeluR2 * (z + kGeluC * z * z * z));
      const float t = s * (1.0f - s);
      f = z * s;
      df = s + (t > 0.0f ? z * t * kGeluR2 * (1.0f + 3.0f * kGeluC * z * z) : 0.0f);
      return;
    }
    default:
      f = z;
      df = 1.0f;
  }
}

// |z| for a scale block's maximum: values that are not finite do not count.  The conversion
// makes them NaN codes whatever the scale (measured: +-inf -> 0x7F / 0xFF, NaN -> 0xFF), so a
// poisoned pre-activation still poisons its gradient.
__device__ __forceinline__ float amax_term(float z) {
  const float m = fabsf(z);
  return m < INFINITY ? m : 0.0f;
}

// The four values that a word of codes and their scale byte stand for.
__device__ __forceinline__ void unpack_ckpt4(uint32_t w, int scale, float z[4]) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  // 2^(scale - 127) as a float: byte 0 lies below the normal range
  const float f = __uint_as_float(scale > 0 ? (uint32_t)scale << 23 : 0x00400000u);
  z[0] = lo[0] * f;
  z[1] = lo[1] * f;
  z[2] = hi[0] * f;
  z[3] = hi[1] * f;
}

}  // namespace moe
