// Grouped linear products and data gradients for a few rows per expert (decode batches, single
// tokens): bound by reading the weights once.
//
// A block of 4 wavefronts takes 64 output columns of one expert and up to 32 of its rows at a
// time; the wavefronts split the reduction into four contiguous parts, each streamed through
// a private ring of LDS steps (no barrier), and their fp32 partial tiles are added in
// wavefront order through LDS before the epilogue.
//   linear: a step is 32 rows of W x 64 columns (4 KiB, whole 128-byte lines), read by the
//           transposing LDS read; three steps deep, two blocks per CU: 120 KiB in flight.
//   dx:     W's rows are the output columns and its columns the reduction, which is the order
//           of the matrix instruction's operand: the weights go straight to registers.
// Measured: one token's 8 experts, 2048 -> 768 (25 MB of weights): 12.5 us a call on buffers that
// take turns, 2.0 TB/s (the kernel alone, 8 calls on the same weights: 10.6 us the fastest, 12.8 on
// average), of which the launch, the first copies and the sums through LDS are 4; 4 rows for each of 64 experts,
// 4096 -> 1408 (738 MB): 129 us, 5.7 TB/s.  8 parts instead of 4: 0.5 us less for the one token, 5
// to 13% more elsewhere.  An expert that holds many of the rows is taken 32 rows at a time by
// up to 8 blocks per 64 columns (512 rows, all on one of 32 experts, 4096 -> 2048: 267 us with one
// block, 49 us; with 128-tiles 48).
#include <algorithm>

#include "grouped.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kStreamRows = 32;
constexpr int kRing = 3;
constexpr int kWaveParts = 4;

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int MODE, bool GATHER>
__global__ __launch_bounds__(64 * kWaveParts) void stream_kernel(const GroupedArgs g) {
  constexpr int kStepBytes = MODE == kLinear ? 4096 + kStreamRows * 64 : 0;
  constexpr int kRingBytes = kWaveParts * kRing * kStepBytes;
  constexpr int kPartBytes = kWaveParts * kStreamRows * kStreamCols * 4;
  __shared__ __align__(1024) char smem[kRingBytes > kPartBytes ? kRingBytes : kPartBytes];
  const int e = blockIdx.y, n0 = blockIdx.x * kStreamCols;
  int lo, hi;
  segment(g.offsets, g.R, e, lo, hi);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int red = MODE == kLinear ? g.K : g.N, ncols = MODE == kDx ? g.K : g.N;
  // blockIdx.z: this block's part of a split reduction, or else its place among the blocks that
  // share an expert's rows
  const int part_z = g.split > 1 ? blockIdx.z : 0;
  const int row_z = g.split > 1 ? 0 : blockIdx.z, row_blocks = g.split > 1 ? 1 : gridDim.z;
  if (lo + row_z * kStreamRows >= hi) return;
  // this wavefront's part of this block's part of the reduction
  const int steps = div_up(red, 32), parts = kWaveParts * g.split;
  const int mine = kWaveParts * part_z + wave;
  const int s0 = (int)((int64_t)steps * mine / parts);
  const int s1 = (int)((int64_t)steps * (mine + 1) / parts);
  const char* const zeros = reinterpret_cast<const char*>(g_zeros);
  const size_t x_ld = 2 * (size_t)red;
  f32x4_t acc[2][4];

  auto rows = [&](auto nm_c, int m0, int nlive) __attribute__((always_inline)) {
    constexpr int NM = decltype(nm_c)::value;
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[m][n] = f32x4_t{};
    // this lane's x row of fragment m: linear (LDS copies): row lane / 4, 64 bytes a row, piece c
    // of row r at c ^ (r >> 2), so that 16 rows at one c cover all banks;
    // dx (registers): row lane % 16, piece lane / 16
    const char* xp[NM];
    const int xr = MODE == kLinear ? lane >> 2 : lane & 15;
    const int xc = MODE == kLinear ? (lane & 3) ^ (xr >> 2) : lane >> 4;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      int row = m0 + min(m * 16 + xr, nlive - 1);
      if constexpr (GATHER) {  // a token outside x: row 0 here, zeros at the end
        const int tk = g.row_token[row];
        row = (unsigned)tk < (unsigned)g.T ? tk : 0;
      }
      xp[m] = (const char*)g.x + row * x_ld + 16 * xc;
    }
    if constexpr (MODE == kLinear) {
      const uint32_t ring = (uint32_t)(uintptr_t)(MOE_LDS char*)smem + wave * kRing * kStepBytes;
      const size_t w_ld = 2 * (size_t)g.N;
      const char* wp[4];
      int wk[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wk[i] = i * 8 + (lane >> 3);
        const int c = ((lane & 7) ^ cols_swizzle<kStreamCols>(wk[i])) * 8;
        wp[i] = (const char*)(g.w + (size_t)e * g.K * g.N + min(n0 + c, g.N - 8)) + wk[i] * w_ld;
      }
      auto copy = [&](int s, int slot) __attribute__((always_inline)) {
        const uint32_t at = __builtin_amdgcn_readfirstlane(ring + slot * kStepBytes);
        const int left = s < s1 ? red - s * 32 : 0;  // behind the part: zeros, never used
#pragma unroll
        for (int i = 0; i < 4; ++i)
          copy_to_lds(wk[i] < left ? wp[i] + (size_t)s * 32 * w_ld : zeros, at + i * 1024);
#pragma unroll
        for (int m = 0; m < NM; ++m)
          copy_to_lds(xc * 8 < left ? xp[m] + (size_t)s * 64 : zeros, at + 4096 + m * 1024);
      };
      for (int i = 0; i < kRing; ++i) copy(s0 + i, i);
      const int k = (lane >> 4) * 8 + ((lane & 15) >> 2);  // W row of the transposing read
      const uint32_t wf = ring + k * 128 + (lane & 1) * 8;
      const int wc = (lane & 3) >> 1, ws = cols_swizzle<kStreamCols>(k);
      const uint32_t xf = ring + 4096 + (lane & 15) * 64 + ((lane >> 4) ^ ((lane & 15) >> 2)) * 16;
      int slot = 0;
      for (int s = s0; s < s1; ++s) {
        wait_vm<(kRing - 1) * (4 + NM)>();
        const uint32_t at = slot * kStepBytes;
        bf16x8_t w[4], x[NM];
#pragma unroll
        for (int n = 0; n < 4; ++n) w[n] = read_cols<64>(wf + at + (((2 * n) ^ ws) + wc) * 16);
#pragma unroll
        for (int m = 0; m < NM; ++m) x[m] = read_rows(xf + at + m * 1024);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the step is read: refill it
        copy(s + kRing, slot);
        slot = slot == kRing - 1 ? 0 : slot + 1;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int n = 0; n < 4; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[n], x[m], acc[m][n], 0, 0, 0);
      }
      wait_vm<0>();
    } else {
      const uint4* wp[4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
        wp[n] = (const uint4*)(g.w + ((size_t)e * g.K + min(n0 + n * 16 + (lane & 15), g.K - 1)) *
                                         g.N) + (lane >> 4);
      // steps in fours: their loads are in flight together
      constexpr int kDeep = 4;
      int s = s0;
      for (; s + kDeep <= s1 && (s + kDeep) * 32 <= red; s += kDeep) {
        u32x4 w[kDeep][4], x[kDeep][NM];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
#pragma unroll
          for (int n = 0; n < 4; ++n)
            w[d][n] = __builtin_nontemporal_load((const u32x4*)(wp[n] + (s + d) * 4));
#pragma unroll
          for (int m = 0; m < NM; ++m) x[d][m] = *(const u32x4*)(xp[m] + (size_t)(s + d) * 64);
        }
        __builtin_amdgcn_sched_barrier(0);  // all of them in flight before the first product
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
#pragma unroll
          for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n)
              acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8_t, w[d][n]), __builtin_bit_cast(bf16x8_t, x[d][m]),
                  acc[m][n], 0, 0, 0);
      }
      for (; s < s1; ++s) {
        const bool in = s * 32 + (lane >> 4) * 8 < red;  // the last, partial step
        const u32x4 zero = {0, 0, 0, 0};
        u32x4 w[4], x[NM];
#pragma unroll
        for (int n = 0; n < 4; ++n) w[n] = in ? *(const u32x4*)(wp[n] + s * 4) : zero;
#pragma unroll
        for (int m = 0; m < NM; ++m) x[m] = in ? *(const u32x4*)(xp[m] + (size_t)s * 64) : zero;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int n = 0; n < 4; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, w[n]), __builtin_bit_cast(bf16x8_t, x[m]), acc[m][n],
                0, 0, 0);
      }
    }
    // the parts' tiles [row][64 columns], added in order
    __syncthreads();  // the rings are read
    float* const part = reinterpret_cast<float*>(smem);
    constexpr int kTile = NM * 16 * kStreamCols;
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n)
        *(f32x4_t*)(part + wave * kTile + (m * 16 + (lane & 15)) * kStreamCols + n * 16 +
                    (lane >> 4) * 4) = acc[m][n];
    __syncthreads();
    for (int i = tid; i < NM * 256; i += 64 * kWaveParts) {  // whole wavefronts
      const int r = i >> 4, c = n0 + (i & 15) * 4;
      f32x4_t v = *(const f32x4_t*)(part + i * 4);
#pragma unroll
      for (int w = 1; w < kWaveParts; ++w) v += *(const f32x4_t*)(part + w * kTile + i * 4);
      const bool in = r < nlive && c < ncols;
      if (g.split > 1) {  // the joining kernel adds the blocks' parts
        if (in) *(f32x4_t*)(g.part + ((size_t)part_z * g.R + m0 + r) * ncols + c) = v;
        continue;
      }
      if constexpr (GATHER) {
        const int tk = g.row_token[m0 + min(r, nlive - 1)];
        if ((unsigned)tk >= (unsigned)g.T) v = f32x4_t{};
      }
      finish4<MODE>(g, e, m0 + r, c, in, v);
    }
    __syncthreads();  // before the next rows' copies
  };
  for (int m0 = lo + row_z * kStreamRows; m0 < hi; m0 += row_blocks * kStreamRows) {
    const int n = min(kStreamRows, hi - m0);
    if (n > 16)
      rows(std::integral_constant<int, 2>{}, m0, n);
    else
      rows(std::integral_constant<int, 1>{}, m0, n);
  }
}

}  // namespace

hipError_t launch_grouped_stream(const GroupedArgs& g, int mode, hipStream_t s) {
  if (mode != kLinear && mode != kDx) return hipErrorInvalidValue;  // no weight gradients here
  // an expert's rows beyond the first 32 go to blocks of their own, which end at once where it has
  // no more (at most 8: later rounds find the weights in the caches)
  const int row_blocks = std::max(1, std::min(8, g.R / (2 * kStreamRows)));
  const dim3 grid(div_up(mode == kDx ? g.K : g.N, kStreamCols), g.E,
                  g.split > 1 ? g.split : row_blocks);
  const dim3 block(64 * kWaveParts);
  if (mode == kDx)
    hipLaunchKernelGGL((stream_kernel<kDx, false>), grid, block, 0, s, g);
  else if (g.row_token)
    hipLaunchKernelGGL((stream_kernel<kLinear, true>), grid, block, 0, s, g);
  else
    hipLaunchKernelGGL((stream_kernel<kLinear, false>), grid, block, 0, s, g);
  return hipGetLastError();
}

}  // namespace moe
