// What the kernels of the grouped products share: operands from their natural bf16 layouts,
// copied to LDS by the load-to-LDS path and fed to 16x16x32 instructions.
//
// A stage is 64 of the reduction.  An operand whose reduction is contiguous in memory
// (kRows: rows x 64 elements, 128 bytes a row) is read from LDS as whole 16-byte pieces; one
// whose reduction is the row index (kCols: 64 rows x C elements) through the transposing LDS
// read, so that neither x, W nor dz is ever transposed or packed in memory:
//   linear   x  kRows    W  kCols        dx   dz kRows   W  kRows        dw   x kCols   dz kCols
//
// Two LDS slots, one barrier per stage, in its middle: by then every wavefront holds the second
// half's fragments in registers, and the copies of the stage after the next go into the slot
// just read.  The copies write lane-consecutive 16-byte pieces, so the bank swizzle is made on
// the source side (which piece of its row a lane fetches):
//   kRows  piece c of row r sits at c ^ f(r), f(r) = ((r >> 1) ^ (r << 2)) & 7: 16 rows at one
//          c cover all 64 banks;
//   kCols  piece c of row k sits at c ^ 2 ((k & 3) | (k >> 3 & m) << 2), m = 3 (256 columns) or
//          1 (128), for 64 columns 2 ((k >> 1 & 1) | (k >> 3 & 1) << 1): the 32-byte pairs
//          that a transposing read takes from rows 8 g + 0 .. 3 of its four lane groups lie in
//          different banks.
//
// The copies are written as inline assembly (they have no register outputs) with explicit
// waits: for the builtin form the compiler waits for every copy in flight before each LDS
// read, which would drain the next stage's.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "act.h"
#include "bf16.h"

namespace moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
#define MOE_LDS __attribute__((address_space(3)))

constexpr int kStage = 64;  // reduction elements per stage
enum OperandMode { kRows = 0, kCols = 1 };

// Source of the pieces outside an operand: 16 zero bytes, valid for every lane.
__device__ __align__(16) const uint32_t g_zeros[4] = {0, 0, 0, 0};

// 16 bytes per lane from base + off (base uniform; ONCE: with the non-temporal hint), or from a
// lane's own address, to the wavefront's 1 KiB at lds (uniform), lane by lane.  m0 carries the
// LDS address; one wait state is required after writing it.
template <bool ONCE = false>
__device__ __forceinline__ void copy_to_lds(const char* base, uint32_t off, uint32_t lds) {
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt"
                 :
                 : "v"(off), "s"(base), "s"(lds)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(off), "s"(base), "s"(lds)
                 : "memory");
}
__device__ __forceinline__ void copy_to_lds(const char* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(src), "s"(lds)
               : "memory");
}
// 4 bytes per lane, to the wavefront's 256 bytes at lds.
__device__ __forceinline__ void copy4_to_lds(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(src), "s"(lds)
               : "memory");
}
// Every copy of this wavefront has landed and every LDS read of it has returned: vmcnt(0)
// lgkmcnt(0) as the builtin, which the compiler takes into account (told nothing, it waited
// once more in the middle of the next copies for a register reloaded long before).
__device__ __forceinline__ void wait_copies() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ int rows_swizzle(int r) { return ((r >> 1) ^ (r << 2)) & 7; }
template <int C>
__device__ __forceinline__ int cols_swizzle(int k) {
  static_assert(C == 64 || C == 128 || C == 256, "");
  if (C == 64) return 2 * (((k >> 1) & 1) | (((k >> 3) & 1) << 1));  // two rows per 256 bytes
  return 2 * ((k & 3) | (((k >> 3) & (C == 256 ? 3 : 1)) << 2));
}

// One operand of a tile: C rows (kRows) or columns (kCols), copied by NT threads.
template <int MODE, int C, int NT>
struct Operand {
  static constexpr int kBytes = C * 2 * kStage;
  static constexpr int kLoads = C * 8 / NT;     // 16-byte pieces per thread and stage
  static constexpr int kPieces = MODE == kRows ? 8 : C / 8;  // per LDS row
  static constexpr int kRowsPerLoad = NT / kPieces;
  // kCols: loads i and i + kKinds take the same piece of rows kKinds * kRowsPerLoad apart
  static constexpr int kKinds = MODE == kCols && C == 256 && kRowsPerLoad == 16 ? 2 : 1;

  // This thread's LDS row in load i and its piece of that row in the source.
  static __device__ __forceinline__ int row_of(int tid, int i) {
    return i * kRowsPerLoad + tid / kPieces;
  }
  static __device__ __forceinline__ int piece_of(int tid, int i) {
    const int r = row_of(tid, i), pos = tid % kPieces;
    return pos ^ (MODE == kRows ? rows_swizzle(r) : cols_swizzle<C>(r));
  }

  // 32-bit source offsets from a uniform base, in few registers.  kRows: that of load 0 and
  // the last live row's (rows behind it repeat it); kCols: one per kind of load (pieces behind
  // the last column repeat the last ones).
  uint32_t off[2];
  __device__ __forceinline__ void set(int tid, uint32_t ld, int last) {
    if constexpr (MODE == kRows) {
      off[0] = (uint32_t)row_of(tid, 0) * ld + 16 * piece_of(tid, 0);
      off[1] = (uint32_t)min(last, C - 1) * ld + 16 * piece_of(tid, 0);
    } else {
#pragma unroll
      for (int i = 0; i < kKinds; ++i)
        off[i] = (uint32_t)row_of(tid, i) * ld + 16 * min(piece_of(tid, i), last);
    }
  }
  __device__ __forceinline__ const char* base_of(const char* base, int i, size_t ld) const {
    return MODE == kRows ? base : base + (size_t)(i / kKinds * kKinds * kRowsPerLoad) * ld;
  }
  __device__ __forceinline__ uint32_t off_of(int i, uint32_t ld) const {
    return MODE == kRows ? min(off[0] + (uint32_t)(i * kRowsPerLoad) * ld, off[1])
                         : off[i % kKinds];
  }
};

// Fragment addresses (bytes from the operand's LDS start) of a lane: kRows: one per half of
// the stage, the fragment's first row added as 128 * row; kCols: one per fragment.
__device__ __forceinline__ uint32_t rows_frag(int lane, int kk) {
  const int r = lane & 15;
  return r * 128 + ((kk * 4 + (lane >> 4)) ^ rows_swizzle(r)) * 16;
}
template <int C>
__device__ __forceinline__ uint32_t cols_frag(int lane, int c0) {  // columns c0 .. c0 + 15
  const int k = (lane >> 4) * 8 + ((lane & 15) >> 2);
  return k * C * 2 + ((c0 / 8) ^ cols_swizzle<C>(k)) * 16 + (lane & 3) * 8;
}
__device__ __forceinline__ bf16x8_t read_rows(uint32_t a) {
  return __builtin_bit_cast(bf16x8_t, *(MOE_LDS const u32x4*)(uintptr_t)a);
}
template <int C>
__device__ __forceinline__ bf16x8_t read_cols(uint32_t a) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(uintptr_t)a);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(uintptr_t)(a + 4 * C * 2));
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Exchanges between the four groups of 16 lanes: two fragments whose lanes hold 4 consecutive
// columns each become one register pair of 8 consecutive columns (lane group g: columns
// swapped_col(g) .. + 7 of the fragments' 32), and back.
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ int swapped_col(int lane) {
  const int g = lane >> 4;
  return (g & 1) * 16 + (g >> 1) * 8;
}
// The maximum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max_groups(float v) {
  uint32_t a = __float_as_uint(v), b = a;
  swap16(a, b);
  const float m = fmaxf(__uint_as_float(a), __uint_as_float(b));
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false,
                                                  false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

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
  int split;    // parts of the reduction; with more than one their sums go to `part`
  float* part;  // linear, dx: [split][R][columns]; dw: [split][E][K][N]
};

// Rows [lo, hi) of expert e, inside [0, R) whatever offsets holds.
__device__ __forceinline__ void segment(const int32_t* offsets, int R, int e, int& lo, int& hi) {
  lo = offsets ? min(max(offsets[e], 0), R) : 0;
  hi = offsets ? max(lo, min(offsets[e + 1], R)) : R;
}

enum GroupedMode { kLinear = 0, kDx = 1, kDw = 2 };

// Which kernel a call takes, chosen from its sizes alone (the row counts are on the device).
enum GroupedKernel { kStream = 0, kTile256, kTile128, kTile64, kTile128Once };
struct GroupedPlan {
  GroupedKernel kernel;
  int split;        // parts of the reduction
  size_t ws_bytes;  // their sums
};
GroupedPlan grouped_plan(const moe_grouped& p, int mode);

// ---- grouped_stream.hip: linear and dx for a few rows per expert
constexpr int kStreamCols = 64;
hipError_t launch_grouped_stream(const GroupedArgs& g, int mode, hipStream_t s);

// Columns c .. c + 3 of row r of linear's or dx's output from its 4 sums v (a 32-column block:
// 8 consecutive lanes, all of them here).
template <int MODE>
__device__ __forceinline__ void finish4(const GroupedArgs& g, int e, int r, int c, bool live,
                                        f32x4_t v) {
  const int ncols = MODE == kDx ? g.K : g.N;
  const size_t o = (size_t)r * ncols + c;
  float y[4];
  if constexpr (MODE == kLinear) {
    float z[4];
    uint2 b = make_uint2(0, 0);
    if (g.bias && live) b = *(const uint2*)(g.bias + (size_t)e * ncols + c);
    z[0] = v[0] + bf16_lo(b.x);
    z[1] = v[1] + bf16_hi(b.x);
    z[2] = v[2] + bf16_lo(b.y);
    z[3] = v[3] + bf16_hi(b.y);
    if (g.codes) {  // uniform
      float m = fmaxf(fmaxf(amax_term(z[0]), amax_term(z[1])),
                      fmaxf(amax_term(z[2]), amax_term(z[3])));
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
      const int ex = ue8m0_exp(m);
      if (live) {
        *(uint32_t*)(g.codes + o) = pack_fp8x4(z, -ex);
        if (c % kQBlock == 0) g.scales[o / kQBlock] = (uint8_t)(ex + 127);
      }
    }
    uint2 q = make_uint2(0, 0);
    if (g.residual && live) q = *(const uint2*)(g.residual + o);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = act_value(g.act, z[i]);
    y[0] += bf16_lo(q.x);
    y[1] += bf16_hi(q.x);
    y[2] += bf16_lo(q.y);
    y[3] += bf16_hi(q.y);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = v[i];
    if (g.codes && live) {
      float z[4], f[4];
      unpack_ckpt4(*(const uint32_t*)(g.codes + o), g.scales[o / kQBlock], z);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float df;
        act_both(g.act, z[i], f[i], df);
        y[i] *= df;
      }
      if (g.a) *(uint2*)(g.a + o) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    }
  }
  if (live) *(uint2*)(g.out + o) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
}

}  // namespace moe
