// Grouped products on microscaled operands (moe_grouped_linear_fp4): weights in 4 bits, x in 4 or
// 8, fp32 accumulation on the scaled matrix cores, epilogue as moe_grouped_linear.
//
// LightLLM PR #1687 (PR body): the expert GEMMs run on the expert prefix-sum layout with block
// scales that are powers of two.
#include <algorithm>

#include "grouped_fp4.h"
#include "moe_internal.h"
#include "wave.h"

namespace moe {
namespace {

constexpr int kXcds = 8;
constexpr int kStageBlocks = 8;  // scale blocks per stage: 256 of the reduction
#define MOE_INLINE __attribute__((always_inline))
#define MOE_LDS __attribute__((address_space(3)))

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// Source of the pieces behind a row's end.
__device__ __align__(16) const uint32_t g_zeros[4] = {0, 0, 0, 0};

// 16 bytes per lane from base + off (base uniform), or from a lane's own address, to the
// wavefront's 1 KiB at lds (uniform), lane by lane; m0 carries the LDS address and needs one wait
// state.  (Inline assembly without register outputs: for the builtin the compiler waits for every
// copy in flight before each LDS read.)
template <bool ONCE = false>  // with the non-temporal hint
__device__ __forceinline__ void copy_to_lds(const uint8_t* base, uint32_t off, uint32_t lds) {
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
__device__ __forceinline__ void copy_to_lds(const uint8_t* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(src), "s"(lds)
               : "memory");
}
// Every copy of this wavefront has landed and every LDS access of it is done (as the builtin,
// which the compiler takes into account).
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
// A basic block of its own where lanes meet again after a divergent branch.
__device__ __forceinline__ void meet() { asm volatile(""); }

// An LDS row holds 128 bytes of an operand's row as eight 16-byte pieces, piece c of row r at
// c ^ f(r): 16 rows at one c cover all banks.  The copies write lane-consecutive pieces, so the
// exchange is made on the source side.
__device__ __forceinline__ int rows_swizzle(int r) { return ((r >> 1) ^ (r << 2)) & 7; }

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// The scale bytes of blocks b .. b + 7 of a row that has nb (see scale_word).
__device__ __forceinline__ u32x2 scale_words(const uint8_t* row, int b, int nb) {
  u32x2 v;
  if (b + 8 <= nb) {
    __builtin_memcpy(&v, row + b, 8);
  } else {
    v[0] = scale_word(row, b, nb);
    v[1] = scale_word(row, b + 4, nb);
  }
  return v;
}

// One output tile, or one part of its reduction.
struct Item {
  int e;       // expert
  int m0;      // first row
  int rows;    // live rows
  int n0;      // first output column
  int part;    // of a split reduction
  int s0, s1;  // its stages
};

// Persistent.  A tile is BM rows of x against 64 WN weight rows: 64 WN output columns, or 32 WN of
// both weight sets (fragment 0 of a wavefront the gate, fragment 1 the factor of the same columns).
// The items are ordered expert by expert, within an expert by groups of 8 M tiles, within a group
// N tile by N tile with the M tiles innermost, and cut into 8 shares of equal cost, one per XCD; a
// block takes every n-th item of its XCD's share, so that neighbours share operand bytes in that
// XCD's L2.
//
// A stage is 256 of the reduction in four steps of one instruction's depth.  Two LDS slots, one
// barrier per stage, before its last step: by then every wavefront holds that step's fragments in
// registers, and the copies of the stage after the next go into the slot just read.  Scale bytes
// come through registers (their rows need not be aligned): loaded with a stage's copies, stored
// before the barrier behind which the stage is read, ordered so that one LDS read brings a lane
// the words of all its fragments.
// ONCE: weight copies with the non-temporal hint, for the calls whose experts have one M tile each on
// the average (fp4_plan).
//
// What it takes: a 256 x 256 tile brings 64 KiB of codes and 4 KiB of scales to LDS per stage, and the
// CUs together draw 10.4 to 11 TB/s from their L2s (a rate reached; that it is their limit has not
// been shown).  Copies alone, without products, take 70 to 80% of the whole time of 16384 x 8192 x
// 8192; an eighth of a scale row's line is used at a time.  3.2 PFLOP/s on ragged rows (131072 rows of
// 256 experts, 7168 -> 2048 twice, 2.4 ms), 4.0 on that dense product; the instruction alone reaches
// 8.2 (fp4, 32 x 32 x 64; 16 x 16 x 128: 6.1) and 4.5 with x in 8 bits.  Few rows per expert: the
// weights' bytes, 5.7 TB/s (1024 rows of 256 experts, 7168 -> 2048 twice: 690 us).  Few stages:
// latency, the first two stages of an item being copied beside the last ones of the item before it.
template <bool EIGHT, bool GATHER, int BM, int WM, int WN, bool ONCE = false>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2)))
void fp4_tile_kernel(const Fp4Args g) {
  constexpr int NT = 64 * WM * WN, BN = 64 * WN;
  constexpr int FM = BM / 32 / WM;            // fragments of a wavefront, by 2
  constexpr int kSubs = EIGHT ? 2 : 1;        // LDS rows per row of x
  constexpr int kRpl = NT / 8;                // LDS rows per load
  constexpr int kA = BM * kSubs / kRpl, kB = BN / kRpl;
  constexpr int kABytes = BM * kSubs * 128, kBBytes = BN * 128;
  constexpr int kScA = kABytes + kBBytes, kScB = kScA + BM * 8;
  constexpr int kSlot = kScB + BN * 8;
  // stages whose scales one load brings, see run
  constexpr int kMost = NT == 512 && !EIGHT && !GATHER ? 4 : 2;
  static_assert(BM % kRpl == 0 && BM + BN <= NT && (kRpl == 64 || kRpl == 32), "");
  __shared__ __align__(1024) char smem[2 * kSlot];
  __shared__ int s_start[kMaxE + 1];  // M tiles before each expert
  __shared__ int s_beg[kMaxE + 1];    // its first row (read from memory for every item: 32.4
                                      // instead of 30.4 us for 2048 rows of 64 experts, 1024 -> 1408)
  __shared__ int s_wsum[WM * WN];
  __shared__ int s_wcost[WM * WN];
  __shared__ int s_share[kXcds + 1];  // first item of each XCD's share

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(MOE_LDS char*)smem;
  const bool gated = g.up.codes != nullptr;
  const int cols = gated ? BN / 2 : BN;  // output columns of a tile
  const int nb = g.K / 32, nst = div_up(nb, kStageBlocks);
  const int ntn = div_up(g.N, cols), per_tile = ntn * g.split;  // items per M tile

  // ---- the M tiles before each expert, and this XCD's share of the items: an eighth of what they
  // cost in rows, a tile's own time being that of 3/4 of its height more than its rows'
  const int xcd = blockIdx.x % kXcds, slots = gridDim.x / kXcds;
  const bool one = g.E == 1;
  int first, last, beg1 = 0, end1 = 0;
  if (one) {
    fp4_segment(g, 0, beg1, end1);
    beg1 = __builtin_amdgcn_readfirstlane(beg1);
    end1 = __builtin_amdgcn_readfirstlane(end1);
    const int total = div_up(end1 - beg1, BM) * per_tile;
    first = (int)((int64_t)total * xcd / kXcds);
    last = (int)((int64_t)total * (xcd + 1) / kXcds);
  } else {
    auto cost_of = [&](int len, int tiles) MOE_INLINE { return len + tiles * (BM * 3 / 4); };
    const int per = div_up(g.E, NT);
    const int e0 = min(g.E, tid * per), e1 = min(g.E, e0 + per);
    int sum = 0, cost = 0, lo = 0, hi = 0;
    for (int e = e0; e < e1; ++e) {
      fp4_segment(g, e, lo, hi);
      const int tiles = div_up(hi - lo, BM);
      sum += tiles;
      cost += cost_of(hi - lo, tiles);
    }
    const int inc = wave_inclusive_scan(sum), cinc = wave_inclusive_scan(cost);
    if (lane == 63) {
      s_wsum[wave] = inc;
      s_wcost[wave] = cinc;
    }
    if (tid <= kXcds) s_share[tid] = 0;
    __syncthreads();
    int base = inc - sum, total = 0, cbase = cinc - cost, ctotal = 0;
    for (int w = 0; w < WM * WN; ++w) {
      if (w < wave) {
        base += s_wsum[w];
        cbase += s_wcost[w];
      }
      total += s_wsum[w];
      ctotal += s_wcost[w];
    }
    for (int e = e0; e < e1; ++e) {
      fp4_segment(g, e, lo, hi);
      const int tiles = div_up(hi - lo, BM);
      const int c = cost_of(hi - lo, tiles);
      s_start[e] = base;
      s_beg[e] = lo;
      for (int q = 1; q < kXcds; ++q) {  // the shares that end inside this expert
        const int at = (int)((int64_t)ctotal * q / kXcds);
        if (at >= cbase && at < cbase + c)
          s_share[q] = base * per_tile + (int)((int64_t)(at - cbase) * (tiles * per_tile) / c);
      }
      base += tiles;
      cbase += c;
    }
    if (tid == NT - 1) {
      s_start[g.E] = total;
      s_beg[g.E] = min(max(g.offsets[g.E], 0), g.R);
      s_share[kXcds] = total * per_tile;
    }
    __syncthreads();
    first = __builtin_amdgcn_readfirstlane(s_share[xcd]);
    last = __builtin_amdgcn_readfirstlane(s_share[xcd + 1]);
  }
  first += (int)blockIdx.x / kXcds;
  auto find = [&](int item) MOE_INLINE {
    Item t;
    int tiles, local, beg, end;  // of the expert: M tiles, the item's place, the rows
    if (one) {
      t.e = 0;
      tiles = div_up(end1 - beg1, BM);
      local = item;
      beg = beg1;
      end = end1;
    } else {
      auto start = [&](int e) MOE_INLINE { return __builtin_amdgcn_readfirstlane(s_start[e]); };
      int lo = 0, hi = g.E;
      const int q = item / per_tile;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start(mid) <= q) lo = mid; else hi = mid;
      }
      t.e = lo;
      tiles = start(lo + 1) - start(lo);
      local = item - per_tile * start(lo);
      beg = s_beg[lo];  // (as fp4_segment)
      end = max(beg, s_beg[lo + 1]);
    }
    constexpr int kGroup = 8;
    const int group = local / (kGroup * per_tile) * kGroup;
    local -= group * per_tile;
    const int in_group = min(kGroup, tiles - group), nt = local / in_group;
    const int mt = group + local - nt * in_group;
    t.part = __builtin_amdgcn_readfirstlane(nt / ntn);
    t.s0 = nst * t.part / g.split;
    t.s1 = nst * (t.part + 1) / g.split;
    // tiles of even height, in steps of a fragment per wavefront row
    const int height = div_up(div_up(end - beg, tiles), 32 * WM) * 32 * WM;
    t.m0 = __builtin_amdgcn_readfirstlane(beg + mt * height);
    t.rows = __builtin_amdgcn_readfirstlane(min(height, end - t.m0));
    t.n0 = __builtin_amdgcn_readfirstlane((nt - t.part * ntn) * cols);
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    return t;
  };

  // ---- copies
  const uint32_t a_ld = EIGHT ? g.K : g.K / 2, b_ld = g.K / 2;
  constexpr int kAStep = 128 * kSubs;  // bytes of a row per stage
  const uint8_t *a_base, *b_base[2];
  const uint8_t* a_ptr[GATHER ? BM / kRpl : 1];
  uint32_t a_off = 0, a_last = 0, b_off = 0, b_last[2] = {0, 0};
  const uint8_t* sc_ptr;  // this thread's row of scales
  // Its words: 0, 1 of the stage whose scales are to be stored next, 2 .. of those after it where
  // two or four were loaded at once
  uint32_t __attribute__((ext_vector_type(2 * kMost))) sc;
  const int pos = tid % 8, piece = pos ^ rows_swizzle(tid / 8);
  const uint32_t b_stride = (gated ? 32 : 64) * b_ld;  // from a wavefront column's rows to the next's
  // the row of scales this thread brings: of A, then of B (a thread behind them one again)
  const int sc_row = tid < BM + BN ? tid : tid - (BM + BN);
  const bool scales_a = __builtin_amdgcn_readfirstlane(sc_row) < BM;  // whole wavefronts
  uint32_t sc_at[2];  // the LDS places of its two words of a stage
  {
    const int t = scales_a ? sc_row : sc_row - BM, r = t & 31, f = t >> 5;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      sc_at[h] = scales_a ? kScA + ((((f % WM) * 2 + h) * 32 + r) * FM + f / WM) * 4
                          : kScB + ((((f / 2) * 2 + h) * 32 + r) * 2 + (f & 1)) * 4;
  }
  auto token_of = [&](int row) MOE_INLINE {  // a token outside x: row 0, zeros in the epilogue
    const int tk = g.row_token[row];
    return (unsigned)tk < (unsigned)g.T ? tk : 0;
  };
  auto setup = [&](const Item& t, int tid) MOE_INLINE {
    if constexpr (GATHER) {
#pragma unroll
      for (int i = 0; i < BM / kRpl; ++i)
        a_ptr[i] = g.x + (size_t)token_of(t.m0 + min(i * kRpl + tid / 8, t.rows - 1)) * a_ld +
                   t.s0 * kAStep + 16 * piece;
    } else {
      a_base = g.x + (size_t)t.m0 * a_ld + t.s0 * kAStep;
      a_off = (uint32_t)(tid / 8) * a_ld + 16 * piece;
      a_last = (uint32_t)(t.rows - 1) * a_ld + 16 * piece;
    }
    const size_t w0 = ((size_t)t.e * g.N + t.n0) * b_ld + t.s0 * 128;
    const bool second = gated || t.n0 + 32 < g.N;  // the odd fragments have rows of their own
    b_base[0] = g.w.codes + w0;
    b_base[1] = gated ? g.up.codes + w0 : g.w.codes + w0 + (second ? 32 * b_ld : 0);
    b_off = (uint32_t)(tid / 8 % 32) * b_ld + 16 * piece;
    const int end = min(g.N - t.n0, BN) - 1;
    b_last[0] = (uint32_t)end * b_ld + 16 * piece;
    b_last[1] = b_last[0] - (!gated && second ? 32 * b_ld : 0);
    if (scales_a) {
      int row = t.m0 + min(sc_row, t.rows - 1);
      if constexpr (GATHER) row = token_of(row);
      sc_ptr = g.xs + (size_t)row * nb;
    } else {
      const int q = sc_row - BM, f = (q >> 5) & 1;
      const int n = t.n0 + (q >> 6) * (gated ? 32 : 64) + (gated ? 0 : 32 * f) + (q & 31);
      sc_ptr = (gated && f ? g.up.scales : g.w.scales) + ((size_t)t.e * g.N + min(n, g.N - 1)) * nb;
    }
  };
  // Load i of A, of B: into the slot at LDS address la (this wavefront's part)
  auto b_src = [&](int i, const uint8_t*& base, uint32_t& off) MOE_INLINE {
    if constexpr (kRpl == 64) {  // 64 LDS rows a load: a wavefront column's two fragments
      const bool f = wave >= WM * WN / 2;
      base = b_base[f];
      off = min(b_off + i * b_stride, b_last[f]);
    } else {
      base = b_base[i & 1];
      off = min(b_off + (i >> 1) * b_stride, b_last[i & 1]);
    }
  };
  auto copy_piece = [&](uint32_t la, int i) MOE_INLINE {
    if (i >= kA) {
      const uint8_t* base;
      uint32_t off;
      b_src(i - kA, base, off);
      copy_to_lds<ONCE>(base, off, la + kABytes + (i - kA) * NT * 16);
    } else {
      const int r = i % (BM / kRpl), sub = i / (BM / kRpl);
      if constexpr (GATHER)
        copy_to_lds(a_ptr[r] + 128 * sub, la + i * NT * 16);
      else
        copy_to_lds(a_base + 128 * sub, min(a_off + r * kRpl * a_ld, a_last), la + i * NT * 16);
    }
  };
  // The last, partial stage: left blocks of it.
  auto copy_piece_tail = [&](uint32_t la, int i, int left) MOE_INLINE {
    const uint8_t* src;
    int at = piece;
    if (i >= kA) {
      const uint8_t* base;
      uint32_t off;
      b_src(i - kA, base, off);
      src = base + off;
      la += kABytes + (i - kA) * NT * 16;
    } else {
      const int r = i % (BM / kRpl), sub = i / (BM / kRpl);
      if constexpr (GATHER)
        src = a_ptr[r] + 128 * sub;
      else
        src = a_base + 128 * sub + min(a_off + r * kRpl * a_ld, a_last);
      if constexpr (EIGHT) at = 4 * sub + (piece >> 1);
      la += i * NT * 16;
    }
    copy_to_lds(at < left ? src : reinterpret_cast<const uint8_t*>(g_zeros), la);
  };
  auto next_stage = [&]() MOE_INLINE {
    if constexpr (GATHER) {
#pragma unroll
      for (int i = 0; i < BM / kRpl; ++i) a_ptr[i] += kAStep;
    } else {
      a_base += kAStep;
    }
    b_base[0] += 128;
    b_base[1] += 128;
  };
  auto slot_lds = [&](int slot) MOE_INLINE {
    return (uint32_t)__builtin_amdgcn_readfirstlane(lds0 + slot * kSlot + wave * 1024);
  };
  auto store_scales = [&](int slot) MOE_INLINE {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *(MOE_LDS uint32_t*)(uintptr_t)(lds0 + slot * kSlot + sc_at[h]) = sc[h];
  };
  // Whether load i brings rows that nm fragments use (of B: always).
  auto needed = [](int i, int nm) MOE_INLINE {
    return i >= kA || i % (BM / kRpl) * kRpl < 32 * WM * nm;
  };

  // The copies run ahead of the arithmetic through this block's items in order: the item being
  // copied, its next stage, its fragment rows.
  int cp_idx = first, cp_stage = 0, cp_end = 0, cp_nm = FM;
  auto begin_copies = [&]() MOE_INLINE {
    int tid_v = tid;  // through an empty statement, see the epilogue
    asm volatile("" : "+v"(tid_v));
    const Item t = find(cp_idx);
    setup(t, tid_v);
    cp_stage = t.s0;
    cp_end = t.s1;
    cp_nm = div_up(t.rows, 32 * WM);
  };
  auto copies_done = [&]() MOE_INLINE {  // a stage was copied
    ++cp_stage;
    next_stage();  // (a branch here would split the stage loop's block)
  };
  auto copies_next = [&]() MOE_INLINE {  // on to the next item where all stages are copied
    if (cp_stage < cp_end || cp_idx >= last) return;
    cp_idx += slots;
    if (cp_idx < last) begin_copies();
  };
  auto copy_any = [&](int slot) MOE_INLINE {
    const uint32_t la = slot_lds(slot);
    const int left = nb - cp_stage * kStageBlocks;
    const u32x2 v = scale_words(sc_ptr, cp_stage * kStageBlocks, nb);
    sc[0] = v[0];
    sc[1] = v[1];
    if (left >= kStageBlocks) {
#pragma unroll
      for (int i = 0; i < kA + kB; ++i)
        if (needed(i, cp_nm)) copy_piece(la, i);
    } else {
#pragma unroll
      for (int i = 0; i < kA + kB; ++i)
        if (needed(i, cp_nm)) copy_piece_tail(la, i, left);
    }
  };

  // ---- compute.  Fragment m of a wavefront is rows 32 (m WM + wm) ..
  const int r32 = lane & 31, h = lane >> 5;
  const int fpos = (EIGHT ? h : 4 * h) ^ rows_swizzle(r32);
  const uint32_t fa = lds0 + (wm * 32 + r32) * 128 + fpos * 16;
  const int bpos = (4 * h) ^ rows_swizzle(r32);
  const uint32_t fb = lds0 + kABytes + (wn * 64 + r32) * 128 + bpos * 16;
  const uint32_t fsa = lds0 + kScA + ((wm * 2 + h) * 32 + r32) * FM * 4;
  const uint32_t fsb = lds0 + kScB + ((wn * 2 + h) * 32 + r32) * 8;
  auto lds16 = [&](uint32_t a) MOE_INLINE { return *(MOE_LDS const u32x4*)(uintptr_t)a; };

  f32x16_t acc[FM][2];
  struct Frags {
    u32x4 a[FM][kSubs];
    u32x4 b[2];
  };
  Frags f0, f1;
  uint32_t sa[FM], sb[2], na[FM], nb_[2];  // scale words of this stage and the next
  auto read_a = [&](Frags& f, uint32_t so, int step, int m) MOE_INLINE {
    const uint32_t at = (fa ^ (step * (EIGHT ? 32 : 16))) + so + m * WM * 4096;
    f.a[m][0] = lds16(at);
    if constexpr (EIGHT) f.a[m][1] = lds16(at + BM * 128);
  };
  auto read_b = [&](Frags& f, uint32_t so, int step, int n) MOE_INLINE {
    f.b[n] = lds16((fb ^ (step * 16)) + so + n * 4096);
  };
  auto read_scales = [&](uint32_t so) MOE_INLINE {
    if constexpr (FM == 4) {
      const u32x4 v = lds16(fsa + so);
#pragma unroll
      for (int m = 0; m < FM; ++m) na[m] = v[m];
    } else if constexpr (FM == 2) {
      const u32x2 v = *(MOE_LDS const u32x2*)(uintptr_t)(fsa + so);
      na[0] = v[0];
      na[FM - 1] = v[1];
    } else {
      na[0] = *(MOE_LDS const uint32_t*)(uintptr_t)(fsa + so);
    }
    const u32x2 v = *(MOE_LDS const u32x2*)(uintptr_t)(fsb + so);
    nb_[0] = v[0];
    nb_[1] = v[1];
  };
  auto use_scales = [&]() MOE_INLINE {
#pragma unroll
    for (int m = 0; m < FM; ++m) sa[m] = na[m];
    sb[0] = nb_[0];
    sb[1] = nb_[1];
  };
  // What step 3 copies: nothing, a stage, a stage with the scales of that and the next 1 or 3.
  enum { kNone, kCopy, kCopy2, kCopy4 };
  // Step S of a stage from `cur`; the fragments of the step after it are read meanwhile (of the
  // next stage behind step 3, with its scales), and with kCopy the copies of a whole stage are
  // issued into the slot that this stage no longer reads.
  auto step = [&](auto s_c, int slot, auto nm_c, auto copy_c) MOE_INLINE {
    constexpr int S = decltype(s_c)::value, NM = decltype(nm_c)::value;
    Frags& cur = S % 2 ? f1 : f0;
    Frags& nxt = S % 2 ? f0 : f1;
    constexpr bool COPY = decltype(copy_c)::value != kNone;
    constexpr int kNext = (S + 1) % 4;
    const uint32_t so = (S == 3 ? slot ^ 1 : slot) * kSlot;
    const uint32_t la = COPY ? slot_lds(slot) : 0;
    if constexpr (decltype(copy_c)::value >= kCopy2)
      __builtin_memcpy(&sc, sc_ptr + cp_stage * kStageBlocks,
                       decltype(copy_c)::value == kCopy2 ? 16 : 32);
    if constexpr (S == 3) read_scales(so);
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      if constexpr (COPY) {
        constexpr int per = (kA + kB + NM - 1) / NM;
#pragma unroll
        for (int q = m * per; q < (m + 1) * per && q < kA + kB; ++q)
          if (needed(q, NM)) copy_piece(la, q);
      }
      if (m == 0) {
        read_b(nxt, so, kNext, 0);
        read_b(nxt, so, kNext, 1);
      }
      read_a(nxt, so, kNext, m);
      const i32x8_t a = EIGHT ? operand8(cur.a[m][0], cur.a[m][kSubs - 1]) : operand4(cur.a[m][0]);
      acc[m][0] = fp4_product<EIGHT, S>(operand4(cur.b[0]), a, acc[m][0], sb[0], sa[m]);
      acc[m][1] = fp4_product<EIGHT, S>(operand4(cur.b[1]), a, acc[m][1], sb[1], sa[m]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // ---- epilogue: element 4 q + i of lane l is column 8 q + 4 h + i of row l % 32 of a fragment
  // pair; after the exchange between the half wavefronts a lane holds 8 consecutive columns.  One
  // copy per activation (a choice per element was 8 us of a 256 x 256 tile's 10).
  auto epilogue_of = [&](const Item& t, int nm, auto act_c) MOE_INLINE {
    constexpr int ACT = decltype(act_c)::value;
    // through an empty statement: otherwise what derives from the lane below is computed before
    // the items' loop and kept in registers through it
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int r32 = lane & 31, h = lane >> 5;
    auto biases = [&](const void* bias, int cf, float* v) MOE_INLINE {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = cf + 8 * q + 4 * h;
        uint2 b = make_uint2(0, 0);
        if (bias && c < g.N) b = *(const uint2*)((const uint16_t*)bias + (size_t)t.e * g.N + c);
        v[4 * q] = bf16_lo(b.x);
        v[4 * q + 1] = bf16_hi(b.x);
        v[4 * q + 2] = bf16_lo(b.y);
        v[4 * q + 3] = bf16_hi(b.y);
      }
    };
    // 32 columns from cf on: act(z + b), times the factors of a second fragment if there are any
    auto columns = [&](int f, int cf, auto gated_c) MOE_INLINE {
      constexpr bool GATED = decltype(gated_c)::value;
      float b[16], ub[16];
      biases(g.w.bias, cf, b);
      if constexpr (GATED) biases(g.up.bias, cf, ub);
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        if (m >= nm) break;
        const int r = (m * WM + wm) * 32 + r32;
        const size_t row = (size_t)(t.m0 + r) * g.N;
        const bool in = r < t.rows;
        bool named = true;  // (a row whose token lies outside x: zeros)
        if constexpr (GATHER)
          named = (unsigned)g.row_token[t.m0 + min(r, t.rows - 1)] < (unsigned)g.T;
#pragma unroll
        for (int p = 0; p < 2; ++p) {  // 16 columns: 8 of a lane's own and of its partner's
          const int c = cf + 16 * p + 8 * h;
          const bool live = in && c < g.N;
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int k = 8 * p + i;
            y[i] = act_value(ACT, (named ? acc[m][f][k] : 0.0f) + b[k]);
            if constexpr (GATED) y[i] *= (named ? acc[m][1][k] : 0.0f) + ub[k];
          }
          if (g.residual) {  // uniform
            uint4 res = make_uint4(0, 0, 0, 0);
            if (live) res = *(const uint4*)(g.residual + row + c);
            swap32(res.x, res.z);
            swap32(res.y, res.w);
            float rf[8];
            unpack8(res, rf);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] += rf[i];
          }
          uint4 o = pack8(y);
          swap32(o.x, o.z);
          swap32(o.y, o.w);
          if (live) *(uint4*)(g.y + row + c) = o;
        }
      }
    };
    if (gated) {
      const int cf = t.n0 + wn * 32;
      if (cf < g.N) columns(0, cf, std::true_type{});
    } else {
      const int cf = t.n0 + wn * 64;
      if (cf < g.N) columns(0, cf, std::false_type{});
      if (cf + 32 < g.N) columns(1, cf + 32, std::false_type{});
    }
  };
  auto epilogue = [&](const Item& t, int nm) MOE_INLINE {
    if (g.split > 1) {  // the sums, for the joining kernel
      int lane = threadIdx.x & 63;
      asm volatile("" : "+v"(lane));
      const size_t width = gated ? 2 * (size_t)g.N : g.N;
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int c0 = t.n0 + (gated ? wn * 32 : wn * 64 + 32 * f) + 4 * (lane >> 5);
        float* const col = g.part + (size_t)t.part * g.R * width + (gated && f ? g.N : 0);
#pragma unroll
        for (int m = 0; m < FM; ++m) {
          if (m >= nm) break;
          const int r = (m * WM + wm) * 32 + (lane & 31);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = c0 + 8 * q;
            const f32x4_t v = {acc[m][f][4 * q], acc[m][f][4 * q + 1], acc[m][f][4 * q + 2],
                               acc[m][f][4 * q + 3]};
            if (r < t.rows && c < g.N) *(f32x4_t*)(col + (t.m0 + r) * width + c) = v;
          }
        }
      }
      return;
    }
    switch (g.act) {
      case MOE_ACT_RELU: epilogue_of(t, nm, std::integral_constant<int, MOE_ACT_RELU>{}); break;
      case MOE_ACT_RELU2: epilogue_of(t, nm, std::integral_constant<int, MOE_ACT_RELU2>{}); break;
      case MOE_ACT_SILU: epilogue_of(t, nm, std::integral_constant<int, MOE_ACT_SILU>{}); break;
      case MOE_ACT_GELU_TANH:
        epilogue_of(t, nm, std::integral_constant<int, MOE_ACT_GELU_TANH>{});
        break;
      default: epilogue_of(t, nm, std::integral_constant<int, MOE_ACT_NONE>{});
    }
  };

  if (first >= last) return;  // block-uniform
  begin_copies();
  copy_any(0);
  wait_copies();  // the scales
  store_scales(0);
  copies_done();
  copies_next();
  if (cp_idx < last) {
    copy_any(1);
    wait_copies();
    store_scales(1);
    copies_done();
  }
  wait_copies();
  block_barrier();
  int slot = 0;
  using No = std::integral_constant<int, kNone>;
  constexpr auto S0 = std::integral_constant<int, 0>{};
  constexpr auto S1 = std::integral_constant<int, 1>{};
  constexpr auto S2 = std::integral_constant<int, 2>{};
  constexpr auto S3 = std::integral_constant<int, 3>{};
  for (int idx = first; idx < last; idx += slots) {
    const Item item = find(idx);
    auto run = [&](auto nm_c) MOE_INLINE {
      constexpr int NM = decltype(nm_c)::value;
#pragma unroll
      for (int m = 0; m < NM; ++m) acc[m][0] = acc[m][1] = f32x16_t{};
      read_scales(slot * kSlot);
      use_scales();
#pragma unroll
      for (int n = 0; n < 2; ++n) read_b(f0, slot * kSlot, 0, n);
#pragma unroll
      for (int m = 0; m < NM; ++m) read_a(f0, slot * kSlot, 0, m);
      // Stages behind whose barrier a whole stage of this same item is copied, without branches and
      // by two: 16 bytes of a row's scales at a time, as every load fetches a line (by one, half of
      // the requests to the L2 were for scales).  By four in the tall tile on rows of 4 bits in
      // order: 16384 x 8192 x 8192 554 us instead of 575.  Not for a short reduction (8 stages: 109
      // and 107 us), and not where the rows are gathered (their pointers leave no registers: 8192
      // rows 1024 -> 4096 60 and 56 us) or hold 8 bits (65536 rows 4096 -> 4096 twice 1031 and 1011).
      const int whole = min(nb / kStageBlocks, cp_end);
      const int fast = cp_idx == idx ? max(whole - cp_stage, 0) / 2 * 2 : 0;
      const int stages = item.s1 - item.s0;
      int s = 0;
      auto stage = [&](auto copy_c) MOE_INLINE {
        step(S0, slot, nm_c, No{});
        step(S1, slot, nm_c, No{});
        step(S2, slot, nm_c, No{});
        wait_copies();
        store_scales(slot ^ 1);
        if constexpr (decltype(copy_c)::value == kCopy) {  // not the first of its load
#pragma unroll
          for (int i = 2; i < 2 * kMost; ++i) sc[i - 2] = sc[i];
        }
        wait_copies();
        block_barrier();
        step(S3, slot, nm_c, copy_c);
        use_scales();
        copies_done();
        slot ^= 1;
      };
      if constexpr (kMost == 4) {
        for (const int fours = nst >= 16 ? fast / 4 * 4 : 0; s < fours; s += 4) {
          stage(std::integral_constant<int, kCopy4>{});
          stage(std::integral_constant<int, kCopy>{});
          stage(std::integral_constant<int, kCopy>{});
          stage(std::integral_constant<int, kCopy>{});
        }
      }
      for (; s < fast; s += 2) {
        stage(std::integral_constant<int, kCopy2>{});
        stage(std::integral_constant<int, kCopy>{});
      }
      // The others: a partial stage, the next item's first ones, or nothing left to copy.
      for (; s < stages; ++s) {
        copies_next();
        step(S0, slot, nm_c, No{});
        step(S1, slot, nm_c, No{});
        step(S2, slot, nm_c, No{});
        // through an empty statement: else the compiler moves the products behind the branches
#pragma unroll
        for (int m = 0; m < NM; ++m) asm volatile("" : "+v"(acc[m][0]), "+v"(acc[m][1]));
        wait_copies();
        store_scales(slot ^ 1);
        wait_copies();
        block_barrier();
        if (cp_idx < last) {
          copy_any(slot);
          copies_done();
        }
        step(S3, slot, nm_c, No{});
        use_scales();
        slot ^= 1;
      }
      epilogue(item, NM);
      meet();
    };
    const int nm = div_up(item.rows, 32 * WM);
    if constexpr (FM == 4) {
      if (nm >= 4) run(std::integral_constant<int, 4>{});
      else if (nm == 3) run(std::integral_constant<int, 3>{});
      else if (nm == 2) run(std::integral_constant<int, 2>{});
      else run(std::integral_constant<int, 1>{});
    } else if constexpr (FM == 2) {
      if (nm >= 2) run(std::integral_constant<int, 2>{});
      else run(std::integral_constant<int, 1>{});
    } else {
      run(std::integral_constant<int, 1>{});
    }
  }
}

int cu_count() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (hipGetDevice(&dev) == hipSuccess &&
        hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && v > 0)
      return std::max(kXcds, v / kXcds * kXcds);
    return 256;
  }();
  return n;
}

// Adds the parts of a split reduction in order and finishes: 4 columns per thread.
__global__ __launch_bounds__(256) void fp4_join_kernel(const Fp4Args g) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int nq = g.N / 4, r = (int)(i / nq), c = (int)(i % nq) * 4;
  int lo, hi;
  fp4_segment(g, 0, lo, hi);
  if (g.offsets) hi = min(max(g.offsets[g.E], 0), g.R);
  if (r < lo || r >= hi) return;  // (rows outside every expert are left alone)
  const bool gated = g.up.codes != nullptr;
  const size_t width = gated ? 2 * (size_t)g.N : g.N, o = r * width + c;
  f32x4_t z = {}, u = {};
  for (int p = 0; p < g.split; ++p) {
    const float* const part = g.part + (size_t)p * g.R * width + o;
    z += *(const f32x4_t*)part;
    if (gated) u += *(const f32x4_t*)(part + g.N);
  }
  int e = 0;
  if ((g.w.bias || g.up.bias) && g.offsets) {  // the expert of row r
    int top = g.E;
    while (top - e > 1) {
      const int mid = (e + top) >> 1;
      if (g.offsets[mid] <= r) e = mid; else top = mid;
    }
  }
  if (g.row_token && (unsigned)g.row_token[r] >= (unsigned)g.T) z = u = f32x4_t{};
  fp4_finish4(g, e, r, c, z, u);
}

template <bool EIGHT, bool GATHER>
void launch_tiles(const Fp4Args& g, Fp4Kernel kernel, hipStream_t s) {
  if (kernel == kTile256)
    hipLaunchKernelGGL((fp4_tile_kernel<EIGHT, GATHER, EIGHT ? 128 : 256, 2, 4>), dim3(cu_count()),
                       dim3(512), 0, s, g);
  else if (kernel == kTile128)
    hipLaunchKernelGGL((fp4_tile_kernel<EIGHT, GATHER, EIGHT ? 64 : 128, 2, 2>),
                       dim3(2 * cu_count()), dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((fp4_tile_kernel<EIGHT, GATHER, EIGHT ? 64 : 128, 2, 2, true>),
                       dim3(2 * cu_count()), dim3(256), 0, s, g);
}

}  // namespace

Fp4Plan fp4_plan(const moe_grouped& p, bool eight, bool gated) {
  const int64_t rows = p.R / p.E, active = std::min(p.E, std::max(p.R, 1));
  const int stages = div_up(p.K, 256), big = eight ? 128 : 256;
  // tiles, with half of the experts that have rows having one more than those need
  auto tiles = [&](int bm, int bn) {
    const int64_t mt = std::max<int64_t>(active, p.R / bm + (p.E > 1 ? active / 2 : 1));
    return mt * div_up(p.N, gated ? bn / 2 : bn);
  };
  const int64_t n256 = tiles(big, 256), n128 = tiles(big / 2, 128);
  // few rows, and few tiles or short reductions: latency.  (16 rows for each of 128 experts, 2048 ->
  // 768 twice: 55 us, tiles 59; 8 for each of 64, 4096 -> 1408 twice: 91 and 79 us.  x in 8 bits: 1 for
  // each of the 128: 40 and 33 us; 4 of one 7168 -> 4096: 15 us, tiles in 4 parts the same, 16 of
  // it 18 and 15.)
  if (rows <= (eight ? 4 : 16) && (n128 < 256 || (!eight && stages <= 8))) return {kStream, 1};
  // (4 bits: 128 rows for each of 64 experts, 4096 -> 1408: 77 us, with 128-tiles 80; 96 rows: 69 and
  // 62, with the non-temporal hint 58.  8 bits: 64 rows 108 and 123 us; 48 rows 97 and 100, with the
  // hint 97.  One 4096 x 2048 x 2048, 128 tiles: 23 and 19 us; 4096 x 7168 x 4096, 256 tiles: 67
  // and 80 us.)
  if (16 * rows > 7 * big && n256 >= 192) return {kTile256, 1};
  // weights that are read once for an expert's one tile: with the non-temporal hint (8 rows for each of
  // 256 experts, 7168 -> 1024 twice: 388 and 358 us).  The average alone is known here: where skewed
  // routing gives some experts several tiles the hint costs.  16384 rows of 256 experts, 7168 -> 2048
  // twice, without and with it: even 908 and 889 us; half of the rows with experts of more than a tile
  // 947 and 1003; nine tenths 666 and 744.  2048 -> 768 twice, 8192 rows of 128: 70 and 68,
  // 69 and 69, 62 and 62.
  if (n128 >= 256) return {8 * rows <= 3 * big ? kTile128Once : kTile128, 1};
  // few tiles: long reductions in parts (128 x 7168 x 4096, 32 tiles: 26 us, in 4 parts 18; 512 rows,
  // 128 tiles: 26.3, in 2 parts 25.6, in 4 28; 1024 x 2048 x 2048: 12, in 2 parts 18)
  return {kTile128, (int)std::max<int64_t>(1, std::min<int64_t>(stages / 7, 256 / n128))};
}

// (for either type of x, with or without a second weight set)
size_t grouped_fp4_ws_bytes(const moe_grouped& p) {
  size_t n = 0;
  for (int v = 0; v < 4; ++v) {
    const int split = fp4_plan(p, v & 1, v >> 1).split;
    if (split > 1) n = std::max(n, align256((size_t)split * p.R * p.N * (v >> 1 ? 8 : 4)));
  }
  return n;
}

hipError_t launch_grouped_fp4(const moe_grouped& p, bool eight, const uint8_t* x_codes,
                              const uint8_t* x_scales, const int32_t* row_token,
                              const int32_t* offsets, const Fp4Weights& w, const Fp4Weights& up,
                              int act, const void* residual, void* y, void* ws, hipStream_t s) {
  const Fp4Plan plan = fp4_plan(p, eight, up.codes != nullptr);
  const Fp4Args g{x_codes, x_scales, row_token, offsets, w, up, (const uint16_t*)residual,
                  (uint16_t*)y, p.R, p.T, p.K, p.N, p.E, act, plan.split, (float*)ws};
  if (plan.kernel == kStream) return launch_fp4_stream(g, eight, s);
  if (eight) {
    if (row_token) launch_tiles<true, true>(g, plan.kernel, s);
    else launch_tiles<true, false>(g, plan.kernel, s);
  } else {
    if (row_token) launch_tiles<false, true>(g, plan.kernel, s);
    else launch_tiles<false, false>(g, plan.kernel, s);
  }
  if (plan.split > 1) {
    const int64_t n = (int64_t)g.R * (g.N / 4);
    hipLaunchKernelGGL(fp4_join_kernel, dim3((unsigned)div_up64(n, 256)), dim3(256), 0, s, g);
  }
  return hipGetLastError();
}

}  // namespace moe
