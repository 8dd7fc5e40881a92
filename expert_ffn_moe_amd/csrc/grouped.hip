// Grouped linear products with their epilogues and gradients (moe_grouped_linear, _dx, _dw,
// moe_activation_backward): bf16 operands from their natural layouts, fp32 accumulation.
//
// LightLLM PR #1687 (PR body): the expert GEMMs run on the expert prefix-sum layout; the row
// count of every expert is data dependent and is read on the device from `offsets`.
//
//   linear  z = x W + b,  y = act(z) + residual, z kept as E4M3 codes with UE8M0 scales
//   dx      dx = (dz W^T) act'(z),  a = act(z)
//   dw      dW = x^T dz,  db = sum of dz
//
// One 64 x 64 output tile per block of 4 wavefronts (32 x 32 each, 16x16x32 bf16 matrix
// instructions), the reduction in steps of 32 through LDS.
#include <algorithm>

#include "act.h"
#include "bf16.h"
#include "moe_internal.h"
#include "wave.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;
constexpr int kStep = 32;
constexpr int kPad = 40;  // LDS row stride in elements: 80 bytes

struct GroupedArgs {
  const uint16_t* x;    // linear, dw: x; dx: dz
  const uint16_t* w;    // linear, dx: W; dw: dz
  const int32_t* row_token;
  const int32_t* offsets;
  const uint16_t* bias;
  const uint16_t* residual;
  uint16_t* out;
  uint16_t* a;
  uint8_t* codes;
  uint8_t* scales;
  float* dw;
  float* dbias;
  int R, T, K, N, E, act, accumulate;
};

// Rows [lo, hi) of expert e, inside [0, R) whatever offsets holds.
__device__ __forceinline__ void segment(const int32_t* offsets, int R, int e, int& lo, int& hi) {
  lo = offsets ? min(max(offsets[e], 0), R) : 0;
  hi = offsets ? max(lo, min(offsets[e + 1], R)) : R;
}

enum GroupedMode { kLinear = 0, kDx = 1, kDw = 2 };

template <int MODE>
__global__ __launch_bounds__(256) void grouped_kernel(const GroupedArgs g) {
  __shared__ uint16_t As[kTile][kPad], Bs[kTile][kPad];
  __shared__ float tile[kTile][kTile + 1];
  __shared__ int s_e, s_row, s_hi;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int cols = MODE == kDx ? g.K : g.N;
  const int n0 = blockIdx.x * kTile;
  int e, m0, m1, k1, lo, hi;  // output rows m0 .. m1, reduction 0 .. k1
  if (MODE == kDw) {
    e = blockIdx.z;
    segment(g.offsets, g.R, e, lo, hi);
    m0 = blockIdx.y * kTile;
    m1 = g.K;
    k1 = hi - lo;
  } else {
    if (tid == 0) {
      int t = blockIdx.y;
      s_e = -1;
      for (int i = 0; i < g.E; ++i) {
        segment(g.offsets, g.R, i, lo, hi);
        const int nt = div_up(hi - lo, kTile);
        if (t < nt) {
          s_e = i;
          s_row = lo + t * kTile;
          s_hi = hi;
          break;
        }
        t -= nt;
      }
    }
    __syncthreads();
    e = s_e;
    if (e < 0) return;  // block-uniform
    m0 = s_row;
    m1 = s_hi;
    lo = 0;
    k1 = MODE == kLinear ? g.K : g.N;
  }
  const size_t wbase = (size_t)e * g.K * g.N;
  f32x4_t acc[2][2] = {};
  for (int k0 = 0; k0 < k1; k0 += kStep) {
    for (int i = tid; i < kTile * kStep; i += 256) {
      uint16_t av = 0, bv = 0;
      if (MODE == kDw) {  // both operands have the reduction as their row
        const int c = i % kTile, k = i / kTile;
        if (k0 + k < k1) {
          const int r = lo + k0 + k;
          const int xr = g.row_token ? g.row_token[r] : r;
          const bool ok = !g.row_token || (unsigned)xr < (unsigned)g.T;
          if (m0 + c < m1 && ok) av = g.x[(size_t)xr * g.K + m0 + c];
          if (n0 + c < cols) bv = g.w[(size_t)r * g.N + n0 + c];
        }
        As[c][k] = av;
        Bs[c][k] = bv;
      } else {
        const int k = i % kStep, c = i / kStep;
        if (k0 + k < k1 && m0 + c < m1) {
          const int r = m0 + c;
          const int xr = g.row_token ? g.row_token[r] : r;
          if (!g.row_token || (unsigned)xr < (unsigned)g.T) av = g.x[(size_t)xr * k1 + k0 + k];
        }
        As[c][k] = av;
        if (MODE == kDx) {
          if (k0 + k < k1 && n0 + c < cols) bv = g.w[wbase + (size_t)(n0 + c) * g.N + k0 + k];
          Bs[c][k] = bv;
        } else {
          const int cn = i % kTile, kn = i / kTile;
          if (k0 + kn < k1 && n0 + cn < cols) bv = g.w[wbase + (size_t)(k0 + kn) * g.N + n0 + cn];
          Bs[cn][kn] = bv;
        }
      }
    }
    __syncthreads();
    // 16x16x32 operands: lane l holds row l % 16, reduction 8 (l / 16) .. + 8
    bf16x8_t a[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = __builtin_bit_cast(
          bf16x8_t, *(const u32x4*)&As[(wave >> 1) * 32 + 16 * i + (lane & 15)][8 * (lane >> 4)]);
      b[i] = __builtin_bit_cast(
          bf16x8_t, *(const u32x4*)&Bs[(wave & 1) * 32 + 16 * i + (lane & 15)][8 * (lane >> 4)]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    __syncthreads();
  }
  // element i of lane l is row 4 (l / 16) + i, column l % 16
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        tile[(wave >> 1) * 32 + 16 * i + 4 * (lane >> 4) + q][(wave & 1) * 32 + 16 * j +
                                                              (lane & 15)] = acc[i][j][q];
  __syncthreads();
  // two threads per 32-column block of a row pair: thread = (row, block)
  for (int i = tid; i < kTile * 2; i += 256) {
    const int r = m0 + (i >> 1), c0 = n0 + (i & 1) * 32;
    if (r >= m1 || c0 >= cols) continue;
    const float* v = &tile[i >> 1][(i & 1) * 32];
    const int nc = min(32, cols - c0);
    const size_t o = (size_t)r * cols + c0;
    if (MODE == kDw) {
      float* d = g.dw + wbase + o;
      for (int c = 0; c < nc; ++c) d[c] = g.accumulate ? d[c] + v[c] : v[c];
    } else if (MODE == kDx) {
      float z[4];
      for (int c = 0; c < nc; ++c) {
        float f = 0.0f, df = 1.0f;
        if (g.codes) {
          if (c % 4 == 0) unpack_ckpt4(*(const uint32_t*)(g.codes + o + c), g.scales[o / kQBlock], z);
          act_both(g.act, z[c % 4], f, df);
          if (g.a) g.a[o + c] = to_bf16(f);
        }
        g.out[o + c] = to_bf16(v[c] * df);
      }
    } else {
      float z[32], amax = 0.0f;
      for (int c = 0; c < nc; ++c) {
        z[c] = v[c] + (g.bias ? bf16_lo(g.bias[(size_t)e * cols + c0 + c]) : 0.0f);
        amax = fmaxf(amax, amax_term(z[c]));
        g.out[o + c] = to_bf16(act_value(g.act, z[c]) + (g.residual ? bf16_lo(g.residual[o + c]) : 0.0f));
      }
      if (g.codes) {
        const int ex = ue8m0_exp(amax);
        g.scales[o / kQBlock] = (uint8_t)(ex + 127);
        for (int c = 0; c < 32; c += 4) *(uint32_t*)(g.codes + o + c) = pack_fp8x4(z + c, -ex);
      }
    }
  }
}

// db[e][n]: one thread per column, rows in order.
__global__ __launch_bounds__(64) void dbias_kernel(const GroupedArgs g) {
  const int e = blockIdx.y, n = blockIdx.x * 64 + threadIdx.x;
  int lo, hi;
  segment(g.offsets, g.R, e, lo, hi);
  if (n >= g.N) return;
  float s = 0.0f;
  for (int r = lo; r < hi; ++r) s += bf16_lo(g.w[(size_t)r * g.N + n]);
  float* d = g.dbias + (size_t)e * g.N + n;
  *d = g.accumulate ? *d + s : s;
}

// One 32-column block per thread.
__global__ __launch_bounds__(256) void act_backward_kernel(
    int64_t nblocks, int kb, const int32_t* __restrict__ live, int act,
    const uint16_t* __restrict__ dy, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, uint16_t* __restrict__ dz, uint16_t* __restrict__ a) {
  if (live) nblocks = min(nblocks, (int64_t)max(*live, 0) * kb);
  for (int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x; b < nblocks;
       b += (int64_t)gridDim.x * 256) {
    for (int c = 0; c < 32; c += 8) {
      float z[8], d[8], f[8];
      unpack_ckpt4(*(const uint32_t*)(codes + b * 32 + c), scales[b], z);
      unpack_ckpt4(*(const uint32_t*)(codes + b * 32 + c + 4), scales[b], z + 4);
      unpack8(*(const uint4*)(dy + b * 32 + c), d);
      for (int i = 0; i < 8; ++i) {
        float df;
        act_both(act, z[i], f[i], df);
        d[i] *= df;
      }
      *(uint4*)(dz + b * 32 + c) = pack8(d);
      if (a) *(uint4*)(a + b * 32 + c) = pack8(f);
    }
  }
}

}  // namespace

hipError_t launch_grouped_linear(const moe_grouped& p, const void* x, const int32_t* row_token,
                                 const int32_t* offsets, const void* w, const void* bias, int act,
                                 const void* residual, void* y, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s) {
  GroupedArgs g{(const uint16_t*)x, (const uint16_t*)w, row_token, offsets, (const uint16_t*)bias,
                (const uint16_t*)residual, (uint16_t*)y, nullptr, codes, scales, nullptr, nullptr,
                p.R, p.T, p.K, p.N, p.E, act, 0};
  hipLaunchKernelGGL(grouped_kernel<kLinear>, dim3(div_up(p.N, kTile), div_up(p.R, kTile) + p.E),
                     dim3(256), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_grouped_dx(const moe_grouped& p, const void* dz, const int32_t* offsets,
                             const void* w, int act, const uint8_t* codes, const uint8_t* scales,
                             void* dx, void* a, hipStream_t s) {
  GroupedArgs g{(const uint16_t*)dz, (const uint16_t*)w, nullptr, offsets, nullptr, nullptr,
                (uint16_t*)dx, (uint16_t*)a, const_cast<uint8_t*>(codes),
                const_cast<uint8_t*>(scales), nullptr, nullptr, p.R, p.T, p.K, p.N, p.E, act, 0};
  hipLaunchKernelGGL(grouped_kernel<kDx>, dim3(div_up(p.K, kTile), div_up(p.R, kTile) + p.E),
                     dim3(256), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_grouped_dw(const moe_grouped& p, const void* x, const int32_t* row_token,
                             const void* dz, const int32_t* offsets, int accumulate, float* dw,
                             float* dbias, hipStream_t s) {
  GroupedArgs g{(const uint16_t*)x, (const uint16_t*)dz, row_token, offsets, nullptr, nullptr,
                nullptr, nullptr, nullptr, nullptr, dw, dbias, p.R, p.T, p.K, p.N, p.E, 0,
                accumulate};
  hipLaunchKernelGGL(grouped_kernel<kDw>, dim3(div_up(p.N, kTile), div_up(p.K, kTile), p.E),
                     dim3(256), 0, s, g);
  if (dbias)
    hipLaunchKernelGGL(dbias_kernel, dim3(div_up(p.N, 64), p.E), dim3(64), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_act_backward(int64_t rows, int cols, const int32_t* live, int act,
                               const void* dy, const uint8_t* codes, const uint8_t* scales,
                               void* dz, void* a, hipStream_t s) {
  const int64_t nblocks = rows * (cols / kQBlock);
  const int grid = (int)std::min<int64_t>(div_up64(nblocks, 256), 8192);
  hipLaunchKernelGGL(act_backward_kernel, dim3(grid), dim3(256), 0, s, nblocks, cols / kQBlock,
                     live, act, (const uint16_t*)dy, codes, scales, (uint16_t*)dz, (uint16_t*)a);
  return hipGetLastError();
}

}  // namespace moe
