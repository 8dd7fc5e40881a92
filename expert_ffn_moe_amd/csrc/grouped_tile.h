// The matrix-core tile of the grouped products: operands from their natural bf16 layouts,
// copied to LDS by the load-to-LDS path and fed to 16x16x32 instructions.
//
// A stage is 64 of the reduction.  An operand whose reduction is contiguous in memory
// (kRows: rows x 64 elements, 128 bytes a row) is read from LDS as whole 16-byte pieces; one
// whose reduction is the row index (kCols: 64 rows x C elements) through the transposing LDS
// read, so that neither x, W nor dz is ever transposed or packed in memory:
//   linear   x  kRows    W  kCols        dx   dz kRows   W  kRows        dw   x kCols   dz kCols
//
// Two LDS slots: a stage's copies are issued when the stage before starts to compute, one
// barrier per stage.  The copies write lane-consecutive 16-byte pieces, so the bank swizzle
// is made on the source side (which piece of its row a lane fetches):
//   kRows  piece c of row r sits at c ^ f(r), f(r) = ((r >> 1) ^ (r << 2)) & 7: 16 rows at one
//          c cover all 64 banks;
//   kCols  piece c of row k sits at c ^ 2 ((k & 3) | (k >> 3 & m) << 2), m = 3 (256 columns) or
//          1 (128): the 32-byte pairs that a transposing read takes from rows 8 g + 0 .. 3 of
//          its four lane groups lie in different banks.
//
// The copies are written as inline assembly (they have no register outputs) with explicit
// waits: for the builtin form the compiler waits for every copy in flight before each LDS
// read, which would drain the next stage's.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

// 16 bytes per lane from base + off (base uniform), or from a lane's own address, to the
// wavefront's 1 KiB at lds (uniform), lane by lane.  m0 carries the LDS address; one wait state
// is required after writing it.
__device__ __forceinline__ void copy_to_lds(const char* base, uint32_t off, uint32_t lds) {
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
// Every copy of this wavefront has landed and every LDS read of it has returned.
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ int rows_swizzle(int r) { return ((r >> 1) ^ (r << 2)) & 7; }
template <int C>
__device__ __forceinline__ int cols_swizzle(int k) {
  return 2 * ((k & 3) | (((k >> 3) & (C >= 256 ? 3 : 1)) << 2));
}

// One operand of a tile: C rows (kRows) or columns (kCols), copied by NT threads.
template <int MODE, int C, int NT>
struct Operand {
  static constexpr int kBytes = C * 2 * kStage;
  static constexpr int kLoads = C * 8 / NT;     // 16-byte pieces per thread and stage
  static constexpr int kPieces = MODE == kRows ? 8 : C / 8;  // per LDS row
  static constexpr int kRowsPerLoad = NT / kPieces;

  // This thread's LDS row in load i and its piece of that row in the source.
  static __device__ __forceinline__ int row_of(int tid, int i) {
    return i * kRowsPerLoad + tid / kPieces;
  }
  static __device__ __forceinline__ int piece_of(int tid, int i) {
    const int r = row_of(tid, i), pos = tid % kPieces;
    return pos ^ (MODE == kRows ? rows_swizzle(r) : cols_swizzle<C>(r));
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
  return __builtin_bit_cast(bf16x8_t, *(MOE_LDS const u32x4*)(a));
}
template <int C>
__device__ __forceinline__ bf16x8_t read_cols(uint32_t a) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(a));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(a + 4 * C * 2));
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

}  // namespace moe
