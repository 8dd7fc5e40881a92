// What the kernels of the grouped product on microscaled operands share.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 weight rows (output columns) by 32 rows of x
// over 64 of the reduction.  Operand layout (checked on the device): lane l, half h = l / 32,
// holds row l % 32; E2M1: values 32 h .. 32 h + 31 in 16 bytes; E4M3: values 16 h .. + 15 and
// 32 + 16 h .. + 15 in 32 bytes; its scale byte is that of values 32 h .. 32 h + 31 in both.
//
// The order of the reduction is free as long as both operands agree.  A stage is 256 values,
// eight scale blocks; step s of its four takes blocks s (half 0) and 4 + s (half 1), so that a
// lane's scale bytes of a stage are one word, byte s for step s, which the instruction selects
// by itself, and its E2M1 codes are 64 consecutive bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "bf16.h"
#include "fp4_launch.h"

namespace moe {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

struct Fp4Args {
  const uint8_t* x;   // [R or T, K / 2] (E2M1) or [R or T, K] (E4M3)
  const uint8_t* xs;  // [R or T, K / 32]
  const int32_t* row_token;
  const int32_t* offsets;
  Fp4Weights w, up;  // up.codes NULL: y = act(x W + b), else that times x U + c
  const uint16_t* residual;
  uint16_t* y;
  int R, T, K, N, E, act;
  int split;    // parts of the reduction; with more than one their sums go to `part`
  float* part;  // [split][R][N], with up [split][R][2 N]: z, then u
};

// Rows [lo, hi) of expert e, inside [0, R) whatever offsets holds.
__device__ __forceinline__ void fp4_segment(const Fp4Args& g, int e, int& lo, int& hi) {
  lo = g.offsets ? min(max(g.offsets[e], 0), g.R) : 0;
  hi = g.offsets ? max(lo, min(g.offsets[e + 1], g.R)) : g.R;
}

template <bool EIGHT, int S>
__device__ __forceinline__ f32x16_t fp4_product(const i32x8_t& w, const i32x8_t& x, f32x16_t acc,
                                                uint32_t ws, uint32_t xs) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc, 4, EIGHT ? 0 : 4, S, (int)ws,
                                                         S, (int)xs);
}
__device__ __forceinline__ i32x8_t operand4(const u32x4& v) {
  i32x8_t r = {};
  r[0] = (int)v[0]; r[1] = (int)v[1]; r[2] = (int)v[2]; r[3] = (int)v[3];
  return r;
}
__device__ __forceinline__ i32x8_t operand8(const u32x4& a, const u32x4& b) {
  i32x8_t r;
  r[0] = (int)a[0]; r[1] = (int)a[1]; r[2] = (int)a[2]; r[3] = (int)a[3];
  r[4] = (int)b[0]; r[5] = (int)b[1]; r[6] = (int)b[2]; r[7] = (int)b[3];
  return r;
}

// The word of scale bytes of blocks b .. b + 3 of a row that has nb; blocks behind the row's end
// get byte 0, a scale that leaves their zero codes zeros.  Rows need not begin at words.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int b, int nb) {
  uint32_t v = 0;
  if (b + 4 <= nb) {
    __builtin_memcpy(&v, row + b, 4);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (b + i < nb) v |= (uint32_t)row[b + i] << (8 * i);
  }
  return v;
}

// Columns c .. c + 3 of row r from the sums z (and u).
__device__ __forceinline__ void fp4_finish4(const Fp4Args& g, int e, int r, int c, f32x4_t z,
                                            f32x4_t u) {
  const size_t o = (size_t)r * g.N + c, b = (size_t)e * g.N + c;
  if (g.w.bias) {
    const uint2 q = *(const uint2*)((const uint16_t*)g.w.bias + b);
    z[0] += bf16_lo(q.x);
    z[1] += bf16_hi(q.x);
    z[2] += bf16_lo(q.y);
    z[3] += bf16_hi(q.y);
  }
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = act_value(g.act, z[i]);
  if (g.up.codes) {
    if (g.up.bias) {
      const uint2 q = *(const uint2*)((const uint16_t*)g.up.bias + b);
      u[0] += bf16_lo(q.x);
      u[1] += bf16_hi(q.x);
      u[2] += bf16_lo(q.y);
      u[3] += bf16_hi(q.y);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= u[i];
  }
  if (g.residual) {
    const uint2 q = *(const uint2*)(g.residual + o);
    y[0] += bf16_lo(q.x);
    y[1] += bf16_hi(q.x);
    y[2] += bf16_lo(q.y);
    y[3] += bf16_hi(q.y);
  }
  *(uint2*)(g.y + o) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
}

// ---- grouped_fp4.hip
enum Fp4Kernel { kStream = 0, kTile256, kTile128, kTile128Once };

// Which kernel a call takes and into how many parts it cuts the reduction, from its sizes alone
// (the row counts are on the device).  Heights are those for x in 4 bits; for 8 they are half.
struct Fp4Plan {
  Fp4Kernel kernel;
  int split;
};
Fp4Plan fp4_plan(const moe_grouped& p, bool eight, bool gated);

// ---- grouped_fp4_stream.hip: a few rows per expert
hipError_t launch_fp4_stream(const Fp4Args& g, bool eight, hipStream_t s);

}  // namespace moe
