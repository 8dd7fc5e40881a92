// bf16 to microscaled 4-bit values and back (LightLLM PR #1687, walkthrough row "Grouped MoE
// kernel support": block scales that are exact powers of two; here with E2M1 codes).  Bound by
// memory: 2 bytes and 0.53 bytes per value.
#include <algorithm>

#include "fp4.h"
#include "fp4_launch.h"
#include "moe_internal.h"
#include "wave.h"

namespace moe {
namespace {

constexpr int kBlock = 32;  // values per scale
constexpr int kPer = 2;     // pieces of 8 values per thread, 256 threads apart

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// Piece i: values 8 i .. 8 i + 7; four lanes hold a block.  16384 x 7168: 47 us, 6.3 TB/s (back 48);
// 1 piece per thread 52, 8 pieces 54.
__global__ __launch_bounds__(256) void quantize_kernel(const uint4* __restrict__ x, int64_t i0,
                                                       int64_t n8, int cols8,
                                                       const int32_t* __restrict__ live,
                                                       uint32_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales) {
  if (live) n8 = min(n8, (int64_t)max(*live, 0) * cols8);
  const int64_t at = i0 + (int64_t)blockIdx.x * (256 * kPer) + threadIdx.x;
  uint4 v[kPer];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    v[p] = make_uint4(0, 0, 0, 0);
    if (at + 256 * p < n8)  // read once: with the hint 47 us, without 50
      v[p] = __builtin_bit_cast(uint4, __builtin_nontemporal_load((const u32x4*)(x + at + 256 * p)));
  }
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int64_t i = at + 256 * p;
    uint32_t m = pair_max8(v[p]);
    m = pair_max(m, dpp_u32<kDppQuadXor1>(m));
    m = pair_max(m, dpp_u32<kDppQuadXor2>(m));
    const int s = fp4_scale(max(m & 0xFFFFu, m >> 16));
    if (i < n8) {
      codes[i] = pack_fp4x8(v[p], s);
      if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)s;
    }
  }
}

__global__ __launch_bounds__(256) void dequantize_kernel(const uint32_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         int64_t i0, int64_t n8, int cols8,
                                                         const int32_t* __restrict__ live,
                                                         uint4* __restrict__ out) {
  if (live) n8 = min(n8, (int64_t)max(*live, 0) * cols8);
  const int64_t at = i0 + (int64_t)blockIdx.x * (256 * kPer) + threadIdx.x;
  uint32_t q[kPer];
  int s[kPer];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    q[p] = 0;
    s[p] = 0;
    if (at + 256 * p < n8) {
      q[p] = codes[at + 256 * p];
      s[p] = scales[(at + 256 * p) >> 2];
    }
  }
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const float f = scale_value(s[p]);
    uint4 o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[p], f, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[p], f, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[p], f, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[p], f, 3));
    if (at + 256 * p < n8) out[at + 256 * p] = o;
  }
}

// Weights [E, K, N] -> [E, N, K] in blocks along K.  A thread takes two columns of one 32-row block, a
// wavefront 256 consecutive bytes of a row; the block's wavefronts take consecutive row blocks, and
// the codes go through LDS so that 16 lanes store 256 consecutive bytes of an output row (stored from
// the registers, 16 bytes each, it took 131 us).  128 of 2048 x 768: 87 us, 5.9 TB/s.
constexpr int kWeightWaves = 16;
__global__ __launch_bounds__(64 * kWeightWaves) void quantize_weights_kernel(
    const uint16_t* __restrict__ w, int K, int N, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
  // piece p of column c at p ^ (c & 15): the lanes of a store lie in different banks
  __shared__ uint4 s_codes[128][kWeightWaves];
  __shared__ uint8_t s_scales[128][kWeightWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int kb0 = blockIdx.x * kWeightWaves, nkb = K / kBlock, n0 = blockIdx.y * 128;
  const size_t e = blockIdx.z;
  if (kb0 + wave < nkb && n0 + 2 * lane < N) {
    const uint32_t* src =
        (const uint32_t*)(w + (e * K + (size_t)(kb0 + wave) * kBlock) * N + n0 + 2 * lane);
    uint32_t v[kBlock];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kBlock; ++i) v[i] = __builtin_nontemporal_load(src + (size_t)i * (N / 2));
#pragma unroll
    for (int i = 0; i < kBlock; ++i) m = pair_max(m, v[i] & 0x7FFF7FFFu);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int s = fp4_scale(c ? m >> 16 : m & 0xFFFFu);
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)  // values 8 j + 2 i and the next, of the pair's low or high half
          p[i] = __builtin_amdgcn_perm(v[8 * j + 2 * i + 1], v[8 * j + 2 * i],
                                       c ? 0x07060302u : 0x05040100u);
        q[j] = pack_fp4x8(make_uint4(p[0], p[1], p[2], p[3]), s);
      }
      const int col = 2 * lane + c;
      s_codes[col][wave ^ (col & 15)] = make_uint4(q[0], q[1], q[2], q[3]);
      s_scales[col][wave] = (uint8_t)s;
    }
  }
  __syncthreads();
  const int p = tid & 15;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int col = half * 64 + (tid >> 4);
    if (kb0 + p >= nkb || n0 + col >= N) continue;
    const size_t row = e * N + n0 + col;
    *(uint4*)(codes + row * (K / 2) + (size_t)(kb0 + p) * 16) = s_codes[col][p ^ (col & 15)];
    scales[row * nkb + kb0 + p] = s_scales[col][p];
  }
}

// fn(first piece, blocks) for launches of fewer than 2^31 threads.
template <class Fn>
hipError_t in_launches(int64_t n8, Fn fn) {
  constexpr int64_t kBlocks = 1 << 20;
  for (int64_t at = 0; at < n8; at += kBlocks * 256 * kPer) {
    fn(at, dim3((unsigned)std::min(div_up64(n8 - at, 256 * kPer), kBlocks)));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_quantize_fp4(const void* x, int64_t rows, int cols, const int32_t* live,
                               uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t n8 = rows * (cols / 8);
  return in_launches(n8, [&](int64_t at, dim3 grid) {
    hipLaunchKernelGGL(quantize_kernel, grid, dim3(256), 0, s, (const uint4*)x, at, n8, cols / 8,
                       live, (uint32_t*)codes, scales);
  });
}

hipError_t launch_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                 int cols, const int32_t* live, void* out, hipStream_t s) {
  const int64_t n8 = rows * (cols / 8);
  return in_launches(n8, [&](int64_t at, dim3 grid) {
    hipLaunchKernelGGL(dequantize_kernel, grid, dim3(256), 0, s, (const uint32_t*)codes, scales,
                       at, n8, cols / 8, live, (uint4*)out);
  });
}

hipError_t launch_quantize_fp4_weights(const void* w, int E, int K, int N, uint8_t* codes,
                                       uint8_t* scales, hipStream_t s) {
  const dim3 grid(div_up(K / kBlock, kWeightWaves), div_up(N, 128), E);
  hipLaunchKernelGGL(quantize_weights_kernel, grid, dim3(64 * kWeightWaves), 0, s,
                     (const uint16_t*)w, K, N, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
