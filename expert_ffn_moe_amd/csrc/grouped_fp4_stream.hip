// Grouped products on 4-bit weights for a few rows per expert: bound by reading the weights once,
// 0.53 bytes each.
//
// A block takes two 32-row fragments of an expert's weights (64 output columns, or 32 of both weight
// sets) and up to 32 of its rows at a time.  The weights' rows are the output columns and hold the
// reduction in order, which is the instruction's operand order: they go straight to registers.
// The block's 4 wavefronts split the reduction into contiguous parts (8: no faster, and 1.5 to 2.3
// times slower from 200 blocks up); their fp32 tiles are added in wavefront order through LDS.
// With fewer rows than experts the blocks are those of the experts that have any, which each
// wavefront counts out from the offsets (2 tokens' 16 of 128 experts: 22 us with a block for every
// expert, 11 us).
//
// One token through 8 of 128 gated experts, 2048 -> 768: 192 blocks, 7 us, of which the 13 MB of
// weights are 2.7 at the rate of a copy; the rest is latency (the offsets, the first loads, two
// stages of the reduction per wavefront, the join), and the call on the host takes longer, 8.
#include <algorithm>

#include "grouped_fp4.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kRows = 32;
constexpr int kParts = 4;

// The n-th expert that has rows (from 0), g.E if there are not so many.
__device__ __forceinline__ int nth_expert(const Fp4Args& g, int n, int lane) {
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int lo = 0, hi = 0;
    if (e0 + lane < g.E) fp4_segment(g, e0 + lane, lo, hi);
    uint64_t some = __ballot(lo < hi);
    const int count = __popcll(some);
    if (n < count) {
      for (; n > 0; --n) some &= some - 1;
      return e0 + __builtin_ctzll(some);
    }
    n -= count;
  }
  return g.E;
}

template <bool EIGHT>
__global__ __launch_bounds__(64 * kParts) void fp4_stream_kernel(const Fp4Args g) {
  __shared__ __align__(16) float part[kParts][kRows][64];
  const bool gated = g.up.codes != nullptr;
  const int n0 = blockIdx.x * (gated ? 32 : 64);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int e = blockIdx.y;
  if (gridDim.y < (unsigned)g.E) {
    e = __builtin_amdgcn_readfirstlane(nth_expert(g, e, lane));
    if (e == g.E) return;  // the same in every wavefront
  }
  int lo, hi;
  fp4_segment(g, e, lo, hi);
  const int r32 = lane & 31, h = lane >> 5;
  const int nb = g.K / 32, stages = div_up(nb, 8);
  const int s0 = stages * wave / kParts, s1 = stages * (wave + 1) / kParts;
  const size_t x_ld = EIGHT ? g.K : g.K / 2;
  const uint8_t* wp[2];
  const uint8_t* ws[2];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const Fp4Weights& q = gated && f ? g.up : g.w;
    const int n = min(n0 + (gated ? 0 : 32 * f) + r32, g.N - 1);
    const size_t row = (size_t)e * g.N + n;
    wp[f] = q.codes + row * (g.K / 2);
    ws[f] = q.scales + row * nb;
  }
  for (int m0 = lo + blockIdx.z * kRows; m0 < hi; m0 += gridDim.z * kRows) {
    const int live = min(kRows, hi - m0);
    int row = m0 + min(r32, live - 1);
    if (g.row_token) {  // a token outside x: row 0 here, zeros at the end
      const int tk = g.row_token[row];
      row = (unsigned)tk < (unsigned)g.T ? tk : 0;
    }
    const uint8_t* xp = g.x + row * x_ld;
    const uint8_t* xs = g.xs + (size_t)row * nb;
    f32x16_t acc[2] = {};
    struct Stage {
      u32x4 w[2][4], x[4][2];
      uint32_t sw[2], sx;
    };
    auto load = [&](Stage& t, int s, auto whole_c) {  // whole: all of its blocks are there
      constexpr bool WHOLE = decltype(whole_c)::value;
      const u32x4 zero = {0, 0, 0, 0};
      const int b0 = 8 * s + 4 * h;  // this lane's first block
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          t.w[f][q] = WHOLE || b0 + q < nb
                          ? *(const u32x4*)(wp[f] + (size_t)(b0 + q) * 16)
                          : zero;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (EIGHT) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int b = 8 * s + 4 * i + q;
            t.x[q][i] = WHOLE || b < nb ? *(const u32x4*)(xp + (size_t)b * 32 + 16 * h) : zero;
          }
        } else {
          t.x[q][0] = WHOLE || b0 + q < nb ? *(const u32x4*)(xp + (size_t)(b0 + q) * 16) : zero;
        }
      }
      if constexpr (WHOLE) {
        __builtin_memcpy(&t.sw[0], ws[0] + b0, 4);
        __builtin_memcpy(&t.sw[1], ws[1] + b0, 4);
        __builtin_memcpy(&t.sx, xs + b0, 4);
      } else {
        t.sw[0] = scale_word(ws[0], b0, nb);
        t.sw[1] = scale_word(ws[1], b0, nb);
        t.sx = scale_word(xs, b0, nb);
      }
    };
    auto multiply = [&](const Stage& t) {
      i32x8_t x[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] = EIGHT ? operand8(t.x[q][0], t.x[q][1]) : operand4(t.x[q][0]);
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        acc[f] = fp4_product<EIGHT, 0>(operand4(t.w[f][0]), x[0], acc[f], t.sw[f], t.sx);
        acc[f] = fp4_product<EIGHT, 1>(operand4(t.w[f][1]), x[1], acc[f], t.sw[f], t.sx);
        acc[f] = fp4_product<EIGHT, 2>(operand4(t.w[f][2]), x[2], acc[f], t.sw[f], t.sx);
        acc[f] = fp4_product<EIGHT, 3>(operand4(t.w[f][3]), x[3], acc[f], t.sw[f], t.sx);
      }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    const int whole = min(s1, nb / 8);
    int s = s0;
    for (; s + 2 <= whole; s += 2) {  // two at a time: their loads are in flight together
      Stage a, b;
      load(a, s, Yes{});
      load(b, s + 1, Yes{});
      __builtin_amdgcn_sched_barrier(0);
      multiply(a);
      multiply(b);
    }
    for (; s < whole; ++s) {
      Stage a;
      load(a, s, Yes{});
      multiply(a);
    }
    if (s < s1) {  // the last, partial stage
      Stage a;
      load(a, s, No{});
      multiply(a);
    }
    // element 4 q + i of lane l: column 8 q + 4 h + i of row l % 32
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t v = {acc[f][4 * q], acc[f][4 * q + 1], acc[f][4 * q + 2], acc[f][4 * q + 3]};
        *(f32x4_t*)&part[wave][r32][32 * f + 8 * q + 4 * h] = v;
      }
    __syncthreads();
    for (int i = tid; i < kRows * (gated ? 8 : 16); i += 64 * kParts) {
      const int r = gated ? i >> 3 : i >> 4, c = (gated ? i & 7 : i & 15) * 4;
      f32x4_t z = {}, u = {};
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        z += *(const f32x4_t*)&part[p][r][c];
        if (gated) u += *(const f32x4_t*)&part[p][r][32 + c];
      }
      if (r >= live || n0 + c >= g.N) continue;
      if (g.row_token && (unsigned)g.row_token[m0 + r] >= (unsigned)g.T) z = u = f32x4_t{};
      fp4_finish4(g, e, m0 + r, n0 + c, z, u);
    }
    __syncthreads();  // before the next rows' sums
  }
}

}  // namespace

hipError_t launch_fp4_stream(const Fp4Args& g, bool eight, hipStream_t s) {
  const int row_blocks = std::max(1, std::min(8, g.R / (2 * kRows)));
  const dim3 grid(div_up(g.N, g.up.codes ? 32 : 64), std::min(g.E, g.R), row_blocks);
  const dim3 block(64 * kParts);
  if (eight) hipLaunchKernelGGL(fp4_stream_kernel<true>, grid, block, 0, s, g);
  else hipLaunchKernelGGL(fp4_stream_kernel<false>, grid, block, 0, s, g);
  return hipGetLastError();
}

}  // namespace moe
