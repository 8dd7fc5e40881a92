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
// Every product is the same tile: C = A B with 16x16x32 instructions, the operand roles and the
// reduction (K, N or an expert's rows) exchanged, and everything elementwise in the epilogue, so
// that z, act(z) and act'(z) never make a trip to memory of their own.  What bounds it:
//   - few rows per expert: reading the weights once (grouped_stream.hip, and 128 x 128 tiles
//     with non-temporal copies: 4 rows for each of 256 experts, 7168 -> 2048: 1.12 ms, 6.6 TB/s);
//   - hundreds of rows: the matrix cores, which 256 x 256 tiles keep at 1.28 PFLOP/s on a dense
//     16384 x 7168 x 4096 (0.93 of a large library product), 0.97 to 1.0 PFLOP/s over 256
//     experts of 512 +- 22 rows with activation and checkpoint (their ragged tiles: 3 x 192 or
//     2 x 256 rows per expert);
//   - in between, the operands' way through L2 into LDS and the first and last stages of short
//     items (256 rows for each of 128 experts, 2048 -> 768: 0.18 ms, 570 TFLOP/s; counters: 1.81
//     GB out of the L2 at 10.0 TB/s, the matrix cores busy 30% of the CUs' busy time);
//   - weight gradients: fp32 stores (128 of 2048 x 768, 805 MB, in 0.26 to 0.28 ms, gathered and
//     with bias sums), which the next item's first wait for copies also waits for;
//   - small calls: the launch and the first copies, 6 us, and 0.27 us per stage of 64.
#include <algorithm>

#include "grouped.h"
#include "grouped_launch.h"
#include "moe_internal.h"
#include "wave.h"

namespace moe {
namespace {

constexpr int kXcds = 8;
#define MOE_INLINE __attribute__((always_inline))

// One output tile, or one part of its reduction.
struct Item {
  int e;     // expert
  int m0;    // linear, dx: first row; dw: first of K
  int rows;  // live rows of the tile
  int n0;    // first output column
  int part;  // of a split reduction
  int k0;    // first of the reduction (dw: a row of the layout)
  int red;   // length of the reduction
};

// A basic block of its own where lanes meet again after a divergent branch: merged with a block
// that joins the paths of the items' loop, it would make the compiler take that loop's
// scalars for divergent.
__device__ __forceinline__ void meet() { asm volatile(""); }

// db[e][n], or a part's sums of it: an item per expert, 64 columns and part of the rows.  8
// threads of 8 columns each take a row, NT / 8 rows at a time, 4 of them in flight per thread;
// the threads' sums are added in order.
template <int NT>
__device__ __forceinline__ void bias_sums(const GroupedArgs& g, float* sums) {
  constexpr int kAt = NT / 8, kPitch = 64 + 1;
  const int tid = threadIdx.x, c = tid % 8 * 8, rl = tid / 8;
  const int blocks = div_up(g.N, 64), items = blocks * g.E * g.split;
  float* const out = g.split > 1 ? g.part + (size_t)g.split * g.E * g.K * g.N : g.dbias;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int q = item / blocks, n0 = (item - q * blocks) * 64;
    const int part = q / g.E, e = q - part * g.E;
    int lo, hi;
    segment(g.offsets, g.R, e, lo, hi);
    const int len = hi - lo;
    hi = lo + (int)((int64_t)len * (part + 1) / g.split);
    lo += (int)((int64_t)len * part / g.split);
    float s[8] = {};
    if (n0 + c < g.N)
      for (int r = lo + rl; r < hi; r += 4 * kAt) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = make_uint4(0, 0, 0, 0);
          if (r + i * kAt < hi) v[i] = *(const uint4*)(g.w + (size_t)(r + i * kAt) * g.N + n0 + c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[8];
          unpack8(v[i], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) s[k] += f[k];
        }
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[rl * kPitch + c + i] = s[i];
    __syncthreads();
    // NT / 64 threads per column, 8 rows each, then their sums
    const int col = tid & 63, k = tid >> 6;
    float v = 0.0f;
    for (int r = 8 * k; r < 8 * k + 8; ++r) v += sums[r * kPitch + col];
    __syncthreads();
    sums[k * kPitch + col] = v;
    __syncthreads();
    if (k == 0 && n0 + col < g.N) {
      v = 0.0f;
      for (int r = 0; r < NT / 64; ++r) v += sums[r * kPitch + col];
      float* const o = out + ((size_t)part * g.E + e) * g.N + n0 + col;
      *o = g.split == 1 && g.accumulate ? *o + v : v;
    }
    __syncthreads();
  }
}

// Persistent.  The items are ordered expert by expert, within an expert by groups of 8 M tiles,
// within a group N tile by N tile (and part by part of a split reduction) with the M tiles
// innermost, and cut into 8 shares of equal cost, one per XCD (workgroups go to XCDs
// round-robin); a block takes every n-th item of its XCD's share, so that the operand bytes that
// neighbouring items share (8 x 4 tiles at a time of a dense product) come from that XCD's L2.
// ONCE: the weights are read once (one M tile per expert), with the non-temporal hint.
template <int MODE, bool GATHER, int BM, int BN, int WM, int WN, bool ONCE = false>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2)))
void tile_kernel(const GroupedArgs g) {
  constexpr int NT = 64 * WM * WN;
  constexpr int FM = BM / 16 / WM, FN = BN / 16 / WN;  // fragments of a wavefront
  static_assert(FM % 4 == 0 && FN % 2 == 0, "tiles cut to quarters, column pairs");
  constexpr int AMODE = MODE == kDw ? kCols : kRows, BMODE = MODE == kDx ? kRows : kCols;
  using A = Operand<AMODE, BM, NT>;
  using B = Operand<BMODE, BN, NT>;
  constexpr int kSlot = A::kBytes + B::kBytes;
  __shared__ __align__(1024) char smem[2 * kSlot];
  __shared__ int s_start[MODE == kDw ? 1 : kMaxE + 1];  // linear, dx: M tiles before each expert
  __shared__ int s_wsum[WM * WN];
  __shared__ int s_wcost[WM * WN];
  __shared__ int s_share[kXcds + 1];  // first item of each XCD's share
  __shared__ __align__(128) char s_stage[WM * WN * 2048];  // the epilogue's, see there
  __shared__ int s_tok[MODE == kDw && GATHER ? WM * WN * 128 : 1];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(MOE_LDS char*)smem;
  const int ncols = MODE == kDx ? g.K : g.N;
  const int ntn = div_up(ncols, BN), per_tile = ntn * g.split;  // items per M tile

  // ---- dw: the bias sums first (in a launch of their own a small call took 5 us more)
  if constexpr (MODE == kDw) {
    if (g.dbias) bias_sums<NT>(g, (float*)smem);
    meet();
  }

  // ---- the M tiles before each expert, and this XCD's share of the items: an eighth of what
  // they cost, in rows (linear, dx: a tile's own time is that of 3/4 of its height more than its
  // rows') or stages (dw: storing a tile takes about 6) of an expert's items
  const int xcd = blockIdx.x % kXcds, slots = gridDim.x / kXcds;
  const bool one = g.E == 1;  // nothing to look up: small dense calls start sooner
  int first, last, beg1 = 0, end1 = 0;
  if (one) {
    segment(g.offsets, g.R, 0, beg1, end1);
    beg1 = __builtin_amdgcn_readfirstlane(beg1);
    end1 = __builtin_amdgcn_readfirstlane(end1);
    const int total = (MODE == kDw ? div_up(g.K, BM) : div_up(end1 - beg1, BM)) * per_tile;
    first = (int)((int64_t)total * xcd / kXcds);
    last = (int)((int64_t)total * (xcd + 1) / kXcds);
  } else {
    const int ntk = div_up(g.K, BM);
    // (at most 2^30 rows and three quarters more)
    auto cost_of = [&](int len, int tiles) MOE_INLINE {
      return MODE == kDw ? div_up(len, kStage) + 6 : len + tiles * (BM * 3 / 4);
    };
    const int per = div_up(g.E, NT);
    const int e0 = min(g.E, tid * per), e1 = min(g.E, e0 + per);
    int sum = 0, cost = 0, lo = 0, hi = 0;
    for (int e = e0; e < e1; ++e) {
      segment(g.offsets, g.R, e, lo, hi);
      const int tiles = MODE == kDw ? ntk : div_up(hi - lo, BM);
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
      if (per > 1) segment(g.offsets, g.R, e, lo, hi);
      const int tiles = MODE == kDw ? ntk : div_up(hi - lo, BM);
      const int c = cost_of(hi - lo, tiles);
      if constexpr (MODE != kDw) s_start[e] = base;
      for (int q = 1; q < kXcds; ++q) {  // the shares that end inside this expert
        const int at = (int)((int64_t)ctotal * q / kXcds);
        if (at >= cbase && at < cbase + c)
          s_share[q] = base * per_tile + (int)((int64_t)(at - cbase) * (tiles * per_tile) / c);
      }
      base += tiles;
      cbase += c;
    }
    if (tid == NT - 1) {
      if constexpr (MODE != kDw) s_start[g.E] = total;
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
      tiles = MODE == kDw ? div_up(g.K, BM) : div_up(end1 - beg1, BM);
      t.e = 0;
      local = item;
    } else if constexpr (MODE == kDw) {
      tiles = div_up(g.K, BM);
      t.e = item / (tiles * per_tile);
      local = item - t.e * tiles * per_tile;
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
    }
    if (one) {
      beg = beg1;
      end = end1;
    } else {
      segment(g.offsets, g.R, t.e, beg, end);
    }
    // a weight gradient over few rows is its output: tile after tile of the same rows of dW
    const int grouped = MODE == kDw && end - beg < 4096 ? 1 : 8;
    const int group = local / (grouped * per_tile) * grouped;
    local -= group * per_tile;
    const int in_group = min(grouped, tiles - group), nt = local / in_group;
    const int mt = group + local - nt * in_group;
    if constexpr (MODE == kDw) {
      t.m0 = mt * BM;
      t.rows = min(BM, g.K - t.m0);
      t.k0 = beg;
      t.red = end - beg;
    } else {
      // an expert's tiles are of even height (in steps of a fragment per wavefront row): their
      // items take the same time and move through the weights together (534 rows as 3 x 192
      // instead of 256 + 256 + 22: the 7168 -> 2048 product 4.7 -> 4.1 ms)
      const int height = div_up(div_up(end - beg, tiles), 16 * WM) * 16 * WM;
      t.m0 = __builtin_amdgcn_readfirstlane(beg + mt * height);
      t.rows = __builtin_amdgcn_readfirstlane(min(height, end - t.m0));
      t.k0 = 0;
      t.red = MODE == kLinear ? g.K : g.N;
    }
    t.part = nt / ntn;
    t.n0 = (nt - t.part * ntn) * BN;
    if (g.split > 1) {  // whole stages per part
      const int stages = div_up(t.red, kStage);
      const int b = (int)((int64_t)stages * t.part / g.split) * kStage;
      t.red = min(t.red, (int)((int64_t)stages * (t.part + 1) / g.split) * kStage) - b;
      t.k0 += b;
    }
    // (known to be uniform: the copies' base addresses have to be scalars)
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.n0 = __builtin_amdgcn_readfirstlane(t.n0);
    t.part = __builtin_amdgcn_readfirstlane(t.part);
    t.k0 = __builtin_amdgcn_readfirstlane(t.k0);
    t.red = __builtin_amdgcn_readfirstlane(t.red);
    return t;
  };

  // ---- copies: each piece is base + 32-bit offset, the base moving on by a stage; gathered
  // rows have an address of their own (linear) or are looked up stage by stage (dw)
  A a{};
  B b{};
  const char *a_base, *b_base;
  const char* a_ptr[MODE == kLinear && GATHER ? A::kLoads : 1];
  int tok_row = 0, tok_par = 0;  // dw: first row of the next stage to be copied, its list
  const char* const zeros = reinterpret_cast<const char*>(g_zeros);
  const size_t a_ld = 2 * (size_t)(MODE == kDx ? g.N : g.K);  // bytes of a row of A
  const size_t b_ld = 2 * (size_t)g.N;
  const size_t a_step = AMODE == kRows ? 2 * kStage : kStage * a_ld;
  const size_t b_step = BMODE == kRows ? 2 * kStage : kStage * b_ld;
  // dw with a gather: the tokens of the next stage's rows, as a copy to a list of this
  // wavefront's own, so that no register waits for them.  Two lists take turns from copy to copy,
  // through the items too: no copy goes to a list that another one in flight writes (behind an
  // item's last whole stage next_stage has started one that nothing reads)
  const uint32_t tok_lds = (uint32_t)(uintptr_t)(MOE_LDS int*)s_tok + wave * 512;
  auto load_tokens = [&]() MOE_INLINE {
    copy4_to_lds(g.row_token + min(tok_row + (int)(threadIdx.x & 63), g.R - 1),
                 __builtin_amdgcn_readfirstlane(tok_lds + tok_par * 256));
  };
  auto token = [&](int i, int tid) MOE_INLINE {
    return *(MOE_LDS const uint32_t*)(uintptr_t)(tok_lds + tok_par * 256 + A::row_of(tid, i) * 4);
  };
  auto token_row = [&](uint32_t tk, int i) MOE_INLINE {  // (without branches: see the stage loop)
    const bool named = tk < (uint32_t)g.T;
    const char* p = a_base + a.off[i % A::kKinds] + (uint64_t)(named ? tk : 0) * (uint32_t)a_ld;
    return named ? p : zeros;
  };
  auto setup = [&](const Item& t, int tid) MOE_INLINE {
    if constexpr (AMODE == kRows)
      a_base = (const char*)g.x + 2 * (size_t)t.k0 + (GATHER ? 0 : t.m0 * a_ld);
    else
      a_base = (const char*)g.x + 2 * (size_t)t.m0 + (GATHER ? 0 : t.k0 * a_ld);
    if constexpr (MODE == kLinear)
      b_base = (const char*)g.w + ((size_t)t.e * g.K + t.k0) * b_ld + 2 * (size_t)t.n0;
    else if constexpr (MODE == kDx)
      b_base = (const char*)g.w + ((size_t)t.e * g.K + t.n0) * b_ld + 2 * (size_t)t.k0;
    else
      b_base = (const char*)g.w + t.k0 * b_ld + 2 * (size_t)t.n0;
    if constexpr (MODE == kLinear && GATHER) {
      // a token outside x reads row 0 here and zeros in the epilogue
#pragma unroll
      for (int i = 0; i < A::kLoads; ++i) {
        const int tk = g.row_token[t.m0 + min(A::row_of(tid, i), t.rows - 1)];
        a_ptr[i] = a_base + ((unsigned)tk < (unsigned)g.T ? tk : 0) * a_ld + 16 * A::piece_of(tid, i);
      }
    } else {
      a.set(tid, MODE == kDw && GATHER ? 0 : (uint32_t)a_ld,
            AMODE == kRows ? t.rows - 1 : (g.K - t.m0) / 8 - 1);
    }
    b.set(tid, (uint32_t)b_ld, BMODE == kRows ? ncols - 1 - t.n0 : (ncols - t.n0) / 8 - 1);
    if constexpr (MODE == kDw && GATHER) {
      tok_row = t.k0;
      tok_par ^= 1;
      load_tokens();
    }
  };
  // Piece i of a whole stage (A's loads, then B's) into the slot at LDS address la (tk: dw with a
  // gather, the piece's token).
  auto copy_piece = [&](uint32_t la, int i, uint32_t tk) MOE_INLINE {
    if (i >= A::kLoads) {
      i -= A::kLoads;
      copy_to_lds<ONCE>(b.base_of(b_base, i, b_ld), b.off_of(i, (uint32_t)b_ld),
                        la + A::kBytes + i * NT * 16);
    } else if constexpr (MODE == kLinear && GATHER) {
      copy_to_lds(a_ptr[i], la + i * NT * 16);
      a_ptr[i] += a_step;
    } else if constexpr (MODE == kDw && GATHER) {
      copy_to_lds(token_row(tk, i), la + i * NT * 16);
    } else {
      copy_to_lds(a.base_of(a_base, i, a_ld), a.off_of(i, (uint32_t)a_ld), la + i * NT * 16);
    }
  };
  // The last, partial stage of a reduction: what lies behind it reads as zeros.
  auto copy_piece_tail = [&](uint32_t la, int i, int left, int tid) MOE_INLINE {
    const char* src;
    int at;
    if (i >= A::kLoads) {
      const int j = i - A::kLoads;
      src = b.base_of(b_base, j, b_ld) + b.off_of(j, (uint32_t)b_ld);
      at = BMODE == kRows ? B::piece_of(tid, j) * 8 : B::row_of(tid, j);
      la += A::kBytes + j * NT * 16;
    } else {
      if constexpr (MODE == kLinear && GATHER)
        src = a_ptr[i];
      else if constexpr (MODE == kDw && GATHER)
        src = token_row(token(i, tid), i);
      else
        src = a.base_of(a_base, i, a_ld) + a.off_of(i, (uint32_t)a_ld);
      at = AMODE == kRows ? A::piece_of(tid, i) * 8 : A::row_of(tid, i);
      la += i * NT * 16;
    }
    copy_to_lds(at < left ? src : zeros, la);
  };
  auto next_stage = [&]() MOE_INLINE {
    if constexpr (!GATHER) a_base += a_step;
    b_base += b_step;
    if constexpr (MODE == kDw && GATHER) {
      tok_row += kStage;
      tok_par ^= 1;
      load_tokens();
    }
  };
  auto slot_lds = [&](int slot) MOE_INLINE {
    return (uint32_t)__builtin_amdgcn_readfirstlane(lds0 + slot * kSlot + wave * 1024);
  };
  // Loads of A that hold live rows when a tile's fragments are cut to nm of FM.
  auto a_loads = [&](int nm) MOE_INLINE { return AMODE == kRows ? div_up(A::kLoads * nm, FM) : A::kLoads; };

  // The copies run two stages ahead of the arithmetic, through this block's items in order: the
  // item being copied, what remains of its reduction (at least 1: an empty one is a stage of
  // zeros), the live length of its partial stage and its fragment count.
  int cp_idx = first, cp_left = 0, cp_tail = 0, cp_nm = FM;
  auto frags_of = [&](int rows) MOE_INLINE {  // fragments that are computed: quarters of FM
    return max(1, div_up(rows, BM / 4)) * (FM / 4);
  };
  auto begin_copies = [&]() MOE_INLINE {
    int tid_v = tid;  // through an empty statement, see the epilogue
    asm volatile("" : "+v"(tid_v));
    const Item t = find(cp_idx);
    setup(t, tid_v);
    cp_left = max(t.red, 1);
    cp_nm = frags_of(t.rows);
    cp_tail = t.red % kStage;
  };
  auto copies_left = [&]() MOE_INLINE { return cp_idx < last; };  // block-uniform
  auto copies_done = [&]() MOE_INLINE {  // a stage was copied
    cp_left -= kStage;
    if (cp_left > 0) next_stage();
  };
  // On to the next item where the last one's stages are all copied.
  auto copies_next = [&]() MOE_INLINE {
    if (cp_left > 0 || cp_idx >= last) return;
    cp_idx += slots;
    if (cp_idx < last) begin_copies();
  };
  // A stage of any kind into a slot.
  auto copy_any = [&](int slot) MOE_INLINE {
    const uint32_t la = slot_lds(slot);
    const int na = a_loads(cp_nm);
    if (cp_left >= kStage) {
#pragma unroll
      for (int i = 0; i < A::kLoads + B::kLoads; ++i)
        if (i < na || i >= A::kLoads)
          copy_piece(la, i, MODE == kDw && GATHER && i < A::kLoads ? token(i, tid) : 0);
    } else {
      int tid_v = tid;
      asm volatile("" : "+v"(tid_v));
#pragma unroll
      for (int i = 0; i < A::kLoads + B::kLoads; ++i)
        if (i < na || i >= A::kLoads) copy_piece_tail(la, i, cp_tail, tid_v);
    }
  };

  // ---- compute.  Fragment m of a wavefront is rows 16 (m WM + wm) ..: a tile with few live
  // rows needs the same number of fragments in every wavefront.
  uint32_t fa[AMODE == kRows ? 2 : FM], fb[BMODE == kRows ? 2 : FN];
  if constexpr (AMODE == kRows) {
    fa[0] = lds0 + rows_frag(lane, 0) + wm * 2048;
    fa[1] = lds0 + rows_frag(lane, 1) + wm * 2048;
  } else {
#pragma unroll
    for (int m = 0; m < FM; ++m) fa[m] = lds0 + cols_frag<BM>(lane, (m * WM + wm) * 16);
  }
  const int wcol = wn * FN * 16;
  if constexpr (BMODE == kRows) {
    fb[0] = lds0 + A::kBytes + rows_frag(lane, 0) + wcol * 128;
    fb[1] = lds0 + A::kBytes + rows_frag(lane, 1) + wcol * 128;
  } else {
#pragma unroll
    for (int n = 0; n < FN; ++n) fb[n] = lds0 + A::kBytes + cols_frag<BN>(lane, wcol + n * 16);
  }
  f32x4_t acc[FM][FN];
  bf16x8_t a0[FM], a1[FM], b0[FN], b1[FN];  // the fragments of a stage's two halves
  auto read_a = [&](uint32_t so, int kk, int m) MOE_INLINE {
    return AMODE == kRows ? read_rows(fa[kk] + so + m * WM * 2048)
                          : read_cols<BM>(fa[m] + so + kk * 64 * BM);
  };
  auto read_b = [&](uint32_t so, int kk, int n) MOE_INLINE {
    return BMODE == kRows ? read_rows(fb[kk] + so + n * 2048)
                          : read_cols<BN>(fb[n] + so + kk * 64 * BN);
  };
  auto mfma_row = [&](int m, const bf16x8_t& av, const bf16x8_t* bv) MOE_INLINE {
#pragma unroll
    for (int n = 0; n < FN; ++n)
      acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[n], av, acc[m][n], 0, 0, 0);
  };
  // First half of a stage; the second half's fragments are read meanwhile, ahead of the last
  // products, so that they are there when the wavefronts meet.
  auto half0 = [&](int slot, auto nm_c) MOE_INLINE {
    constexpr int NM = decltype(nm_c)::value, kReads = FN + NM;
    const uint32_t so = slot * kSlot;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
#pragma unroll
      for (int q = m * kReads / NM; q < (m + 1) * kReads / NM; ++q) {
        if (q < FN) b1[q] = read_b(so, 1, q);
        else a1[q - FN] = read_a(so, 1, q - FN);
      }
      mfma_row(m, a0[m], b0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Second half, with the copies of a whole stage into the slot just read (copy_c) and the first
  // half's fragments of the next stage between the products (an item's last stage reads what
  // the next item reads again).
  auto half1 = [&](int slot, auto nm_c, auto copy_c) MOE_INLINE {
    constexpr int NM = decltype(nm_c)::value;
    constexpr int NA = AMODE == kRows ? (A::kLoads * NM + FM - 1) / FM : A::kLoads, NC = NA + B::kLoads;
    const uint32_t so = (slot ^ 1) * kSlot;
    const uint32_t la = slot_lds(slot);
    constexpr bool kTokens = MODE == kDw && GATHER && decltype(copy_c)::value;
    uint32_t tk[A::kLoads] = {};
    if constexpr (kTokens) {
#pragma unroll
      for (int i = 0; i < A::kLoads; ++i) tk[i] = token(i, tid);
    }
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      if constexpr (decltype(copy_c)::value) {
        constexpr int per = (NC + NM - 1) / NM;
#pragma unroll
        for (int q = m * per; q < (m + 1) * per && q < NC; ++q) {
          // with tokens B's loads first, so that they have arrived
          const int i = kTokens ? (q < B::kLoads ? A::kLoads + q : q - B::kLoads)
                                : (q < NA ? q : q - NA + A::kLoads);
          copy_piece(la, i, tk[i < A::kLoads ? i : 0]);
        }
      }
      mfma_row(m, a1[m], b1);
      if (m == 0) {
#pragma unroll
        for (int n = 0; n < FN; ++n) b0[n] = read_b(so, 0, n);
      }
      a0[m] = read_a(so, 0, m);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // ---- epilogue: the columns are the instruction's rows, so a lane holds 4 consecutive
  // columns n0 + wcol + 16 n + 4 (lane / 16) .. + 3 of row lane % 16 of each fragment.
  auto epilogue = [&](const Item& t, int nm) MOE_INLINE {
    // through an empty statement: otherwise what derives from the lane below is computed
    // before the items' loop and kept in registers through it
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int c4 = t.n0 + wcol + 4 * (lane >> 4);
    if (MODE == kDw || g.split > 1) {
      // fp32: the weight gradients, or a part's sums for the joining kernel.  Straight from the
      // registers a store instruction would write 64 bytes of each of 16 rows; through 2 KiB of
      // LDS of the wavefront's own (laid out like a kRows operand: 16 rows x 128 bytes) it
      // writes whole 128-byte lines (dW of 128 experts 2048 x 768, 805 MB: 274 -> 246 us, with
      // the non-temporal hint 192 us).
      const size_t row0 = MODE == kDw ? ((size_t)t.part * g.E + t.e) * g.K + t.m0
                                      : (size_t)t.part * g.R + t.m0;
      const int lr = lane >> 3, c = t.n0 + wcol + (lane & 7) * 4;
      float* const base = (g.split > 1 ? g.part : g.dw) + row0 * ncols + c;
      const bool add = MODE == kDw && g.split == 1 && g.accumulate;
      const uint32_t st = (uint32_t)(uintptr_t)(MOE_LDS char*)s_stage + wave * 2048;
      const int fr = lane & 15, fs = rows_swizzle(fr);
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        if (m >= nm) break;
#pragma unroll
        for (int n = 0; n < FN; n += 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *(MOE_LDS f32x4_t*)(uintptr_t)(st + fr * 128 + (((h * 4 + (lane >> 4)) ^ fs) * 16)) =
                acc[m][n + h];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int lrow = h * 8 + lr, r = (m * WM + wm) * 16 + lrow;
            f32x4_t v = *(MOE_LDS const f32x4_t*)(uintptr_t)(
                st + lrow * 128 + (((lane & 7) ^ rows_swizzle(lrow)) * 16));
            if (r < t.rows && c + 16 * n < ncols) {
              float* const o = base + (size_t)r * ncols + 16 * n;
              if (add) v += *(const f32x4_t*)o;
              // the gradients are written once and are far larger than the caches; a part's
              // sums are read again at once
              if (MODE == kDw && g.split == 1)
                __builtin_nontemporal_store(v, (f32x4_t*)o);
              else
                *(f32x4_t*)o = v;
            }
          }
        }
      }
      return;
    }
    if constexpr (MODE != kDw) {
      const int c8 = t.n0 + wcol + swapped_col(lane);  // after the exchange
      uint2 bias[FN];
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        bias[n] = make_uint2(0, 0);
        if (MODE == kLinear && g.bias && c4 + 16 * n < ncols)
          bias[n] = *(const uint2*)(g.bias + (size_t)t.e * ncols + c4 + 16 * n);
      }
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        if (m >= nm) break;
        const int r = (m * WM + wm) * 16 + (lane & 15);
        const size_t row = (size_t)(t.m0 + r) * ncols;
        bool named = true;
        if constexpr (GATHER)
          named = (unsigned)g.row_token[t.m0 + min(r, t.rows - 1)] < (unsigned)g.T;
#pragma unroll
        for (int n = 0; n < FN; n += 2) {
          const int c = c8 + 16 * n;
          const bool live = r < t.rows && c < ncols;
          float v[8], y[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = named ? acc[m][n][i] : 0.0f;
            v[4 + i] = named ? acc[m][n + 1][i] : 0.0f;
          }
          if constexpr (MODE == kLinear) {
            v[0] += bf16_lo(bias[n].x); v[1] += bf16_hi(bias[n].x);
            v[2] += bf16_lo(bias[n].y); v[3] += bf16_hi(bias[n].y);
            v[4] += bf16_lo(bias[n + 1].x); v[5] += bf16_hi(bias[n + 1].x);
            v[6] += bf16_lo(bias[n + 1].y); v[7] += bf16_hi(bias[n + 1].y);
            if (g.codes) {
              // the fragment pair is one scale block of its row, spread over 4 lanes
              float amax = 0.0f;
#pragma unroll
              for (int i = 0; i < 8; ++i) amax = fmaxf(amax, amax_term(v[i]));
              const int ex = ue8m0_exp(max_groups(amax));
              uint32_t q0 = pack_fp8x4(v, -ex), q1 = pack_fp8x4(v + 4, -ex);
              swap16(q0, q1);
              if (live) {
                *(uint2*)(g.codes + row + c) = make_uint2(q0, q1);
                if (lane < 16) g.scales[(row + c) / kQBlock] = (uint8_t)(ex + 127);
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = act_value(g.act, v[i]);
            if (g.residual) {
              uint4 q = make_uint4(0, 0, 0, 0);
              if (live) q = *(const uint4*)(g.residual + row + c);
              swap16(q.x, q.z);
              swap16(q.y, q.w);
              float f[8];
              unpack8(q, f);
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] += f[i];
            }
          } else {
            if (g.codes) {
              uint2 q = make_uint2(0, 0);
              int sc = 127;
              if (live) {
                q = *(const uint2*)(g.codes + row + c);
                sc = g.scales[(row + c) / kQBlock];
              }
              swap16(q.x, q.y);
              float z[8], f[8];
              unpack_ckpt4(q.x, sc, z);
              unpack_ckpt4(q.y, sc, z + 4);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float df;
                act_both(g.act, z[i], f[i], df);
                y[i] = v[i] * df;
              }
              if (g.a) {
                uint4 o = pack8(f);
                swap16(o.x, o.z);
                swap16(o.y, o.w);
                if (live) *(uint4*)(g.a + row + c) = o;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = v[i];
            }
          }
          uint4 o = pack8(y);
          swap16(o.x, o.z);
          swap16(o.y, o.w);
          if (live) *(uint4*)(g.out + row + c) = o;
        }
        if constexpr (MODE == kDx) __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  if (first >= last) return;  // block-uniform
  begin_copies();
  if constexpr (MODE == kDw && GATHER) wait_copies();  // the first tokens
  copy_any(0);
  copies_done();
  copies_next();
  if (copies_left()) {
    if constexpr (MODE == kDw && GATHER) wait_copies();
    copy_any(1);
    copies_done();
  }
  wait_copies();
  block_barrier();
  int slot = 0;
  using Yes = std::true_type;
  using No = std::false_type;
  for (int idx = first; idx < last; idx += slots) {
    const Item cur = find(idx);
    const int nst = max(1, div_up(cur.red, kStage));
    auto run = [&](auto nm_c) MOE_INLINE {
      constexpr int NM = decltype(nm_c)::value;
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[m][n] = f32x4_t{};
#pragma unroll
      for (int n = 0; n < FN; ++n) b0[n] = read_b(slot * kSlot, 0, n);
#pragma unroll
      for (int m = 0; m < NM; ++m) a0[m] = read_a(slot * kSlot, 0, m);
      // Stages whose mid-point copies a whole stage of this same item: a loop without branches,
      // which the register allocator needs (with one it kept two sets of accumulators).
      const int fast = cp_idx == idx ? max(cp_left, 0) / kStage : 0;
      int s = 0;
      // The loop's addresses pass through an empty statement: one that was spilled is reloaded,
      // and waited for, here and not in the loop, where the wait would be for the copies too.
#pragma unroll
      for (uint32_t& v : fa) asm volatile("" : "+v"(v));
#pragma unroll
      for (uint32_t& v : fb) asm volatile("" : "+v"(v));
      if constexpr (!(MODE == kLinear && GATHER))
        asm volatile("" : "+v"(a.off[0]), "+v"(a.off[1]));
      asm volatile("" : "+v"(b.off[0]), "+v"(b.off[1]));
      for (; s < fast; ++s) {
        half0(slot, nm_c);
        wait_copies();
        block_barrier();
        half1(slot, nm_c, Yes{});
        cp_left -= kStage;
        next_stage();
        slot ^= 1;
      }
      // The others: a partial stage, the next item's first ones, or nothing left to copy.
      for (; s < nst; ++s) {
        copies_next();
        half0(slot, nm_c);
        wait_copies();
        block_barrier();
        if (copies_left()) {
          copy_any(slot);
          copies_done();
        }
        half1(slot, nm_c, No{});
        slot ^= 1;
      }
      if (cur.n0 + wcol < ncols) epilogue(cur, NM);
      meet();
    };
    const int nm = frags_of(cur.rows);
    if (nm == FM)
      run(std::integral_constant<int, FM>{});
    else if (nm == 3 * FM / 4)
      run(std::integral_constant<int, 3 * FM / 4>{});
    else if (nm == FM / 2)
      run(std::integral_constant<int, FM / 2>{});
    else
      run(std::integral_constant<int, FM / 4>{});
  }
}

// 8 columns per thread, from value 8 i0 on: bound by memory, 7.03 bytes per value with a (13400 x
// 1408, 132 MB: 26.8 us a call on buffers that take turns, 4.9 TB/s, the rate of a large copy; 22 us
// for the fastest of 8 on the same buffers, part of it from the last-level cache).
__global__ __launch_bounds__(256) void act_backward_kernel(
    int64_t i0, int64_t n8, int cols8, const int32_t* __restrict__ live, int act,
    const uint4* __restrict__ dy, const uint2* __restrict__ codes,
    const uint8_t* __restrict__ scales, uint4* __restrict__ dz, uint4* __restrict__ a) {
  if (live) n8 = min(n8, (int64_t)max(*live, 0) * cols8);
  const int64_t i = i0 + (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const uint2 q = codes[i];
  const int s = scales[i >> 2];
  const uint4 y = dy[i];
  float z[8], d[8], f[8];
  unpack_ckpt4(q.x, s, z);
  unpack_ckpt4(q.y, s, z + 4);
  unpack8(y, d);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float df;
    act_both(act, z[k], f[k], df);
    d[k] *= df;
  }
  dz[i] = pack8(d);
  if (a) a[i] = pack8(f);
}

// Adds the parts of a split linear or dx in order and finishes: 4 columns per thread, a row's
// 32-column blocks in 8 consecutive lanes.
template <int MODE>
__global__ __launch_bounds__(256) void join_kernel(const GroupedArgs g) {
  const int ncols = MODE == kDx ? g.K : g.N, nq = div_up(ncols, 32) * 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int r = (int)(i / nq), c = (int)(i % nq) * 4;
  int lo, hi;
  segment(g.offsets, g.R, 0, lo, hi);
  const int first = lo;  // rows outside every expert are left alone
  if (g.offsets) hi = min(max(g.offsets[g.E], 0), g.R);
  const bool live = r >= first && r < hi && c < ncols;
  f32x4_t v = {};
  int e = 0;
  if (live) {
    const size_t o = (size_t)r * ncols + c, plane = (size_t)g.R * ncols;
    for (int p = 0; p < g.split; ++p) v += *(const f32x4_t*)(g.part + p * plane + o);
    if (MODE == kLinear && g.bias && g.offsets) {  // the expert of row r
      int top = g.E;
      while (top - e > 1) {
        const int mid = (e + top) >> 1;
        if (g.offsets[mid] <= r) e = mid; else top = mid;
      }
    }
    if (MODE == kLinear && g.row_token && (unsigned)g.row_token[r] >= (unsigned)g.T) v = f32x4_t{};
  }
  finish4<MODE>(g, e, r, c, live, v);
}

// dw and dbias = the parts of a split weight gradient, added in order (n4, nb4: groups of 4).
__global__ __launch_bounds__(256) void join_dw_kernel(const GroupedArgs g, int64_t n4, int64_t nb4,
                                                      const float* bias_part) {
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool bias = i >= n4;
  if (bias) i -= n4;
  if (bias && i >= nb4) return;
  const int64_t n = bias ? nb4 : n4;
  const f32x4_t* const part = (const f32x4_t*)(bias ? bias_part : g.part) + i;
  f32x4_t* const o = (f32x4_t*)(bias ? g.dbias : g.dw) + i;
  f32x4_t v = g.accumulate ? *o : f32x4_t{};
  for (int p = 0; p < g.split; ++p) v += part[p * n];
  *o = v;
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

template <int MODE, bool GATHER>
void launch_tiles(const GroupedArgs& g, GroupedKernel kernel, hipStream_t s) {
  if (kernel == kTile256)
    hipLaunchKernelGGL((tile_kernel<MODE, GATHER, 256, 256, 2, 4>), dim3(cu_count()), dim3(512), 0,
                       s, g);
  else if (kernel == kTile128)
    hipLaunchKernelGGL((tile_kernel<MODE, GATHER, 128, 128, 2, 2>), dim3(2 * cu_count()),
                       dim3(256), 0, s, g);
  else if (MODE != kDw && kernel == kTile128Once)
    hipLaunchKernelGGL((tile_kernel<MODE, GATHER, 128, 128, 2, 2, MODE != kDw>),
                       dim3(2 * cu_count()), dim3(256), 0, s, g);
  else  // (of three blocks per CU two are resident, 57 to 62 KB of LDS each; the others follow)
    hipLaunchKernelGGL((tile_kernel<MODE, GATHER, 64, 128, 1, 4>), dim3(3 * cu_count()), dim3(256),
                       0, s, g);
}

hipError_t run_grouped(const moe_grouped& p, GroupedArgs g, int mode, void* ws, hipStream_t s) {
  const GroupedPlan plan = grouped_plan(p, mode);
  g.split = plan.split;
  g.part = plan.split > 1 ? static_cast<float*>(ws) : nullptr;
  float* const bias_part =
      plan.split > 1 && mode == kDw ? g.part + (size_t)plan.split * g.E * g.K * g.N : nullptr;
  if (plan.kernel == kStream) {
    const hipError_t err = launch_grouped_stream(g, mode, s);
    if (err != hipSuccess) return err;
  } else if (mode == kLinear) {
    if (g.row_token) launch_tiles<kLinear, true>(g, plan.kernel, s);
    else launch_tiles<kLinear, false>(g, plan.kernel, s);
  } else if (mode == kDx) {
    launch_tiles<kDx, false>(g, plan.kernel, s);
  } else {
    if (g.row_token) launch_tiles<kDw, true>(g, plan.kernel, s);
    else launch_tiles<kDw, false>(g, plan.kernel, s);
  }
  if (plan.split > 1) {
    if (mode == kDw) {
      const int64_t n4 = (int64_t)g.E * g.K * g.N / 4;
      const int64_t nb4 = g.dbias ? (int64_t)g.E * g.N / 4 : 0;
      hipLaunchKernelGGL(join_dw_kernel, dim3((unsigned)div_up64(n4 + nb4, 256)), dim3(256), 0, s,
                         g, n4, nb4, bias_part);
    } else {
      const int64_t n = (int64_t)g.R * div_up(mode == kDx ? g.K : g.N, 32) * 8;
      const dim3 grid((unsigned)div_up64(n, 256));
      if (mode == kLinear) hipLaunchKernelGGL(join_kernel<kLinear>, grid, dim3(256), 0, s, g);
      else hipLaunchKernelGGL(join_kernel<kDx>, grid, dim3(256), 0, s, g);
    }
  }
  return hipGetLastError();
}

}  // namespace

GroupedPlan grouped_plan(const moe_grouped& p, int mode) {
  GroupedPlan plan{kTile64, 1, 0};
  const int ncols = mode == kDx ? p.K : p.N, red = mode == kLinear ? p.K : p.N;
  const int64_t rows = p.R / p.E, active = std::min(p.E, std::max(p.R, 1));
  // tiles, with half of the experts having one more than their rows need
  auto tiles = [&](int bm, int bn) -> int64_t {
    const int64_t mt = mode == kDw ? (int64_t)p.E * div_up(p.K, bm)
                                   : std::max<int64_t>(active, p.R / bm + (p.E > 1 ? p.E / 2 : 1));
    return mt * div_up(ncols, bn);
  };
  const int64_t n256 = tiles(256, 256), n128 = tiles(128, 128), n64 = tiles(64, 128);
  const int64_t stream = active * div_up(ncols, kStreamCols);
  auto parts = [](int64_t a, int64_t b) { return (int)std::max<int64_t>(1, std::min(a, b)); };
  if (mode == kDw) {
    // 256-tiles where they fill the chip (2048 x 768 x 128 experts: 192 us against 221 us with
    // 128-tiles); else over many rows 128-tiles and the rows split (one 2048 x 768 over 16384
    // rows: 131 -> 65 us with 5 parts; over 3000 rows 25 us, 64-tiles 28; over 1536 rows 21 us
    // with 3 parts, 64-tiles 13); over fewer rows the smallest that fill it
    if (n256 >= 192) {
      plan.kernel = kTile256;
    } else if (rows >= 2048) {
      plan.kernel = kTile128;
      plan.split = parts(rows / 512, 512 / n128);
    } else if (n128 >= 256) {
      plan.kernel = kTile128;
    }
  } else if (p.R <= 16 * (int64_t)p.E && stream <= (mode == kDx ? 512 : 1536)) {
    // few rows, few weights: latency.  (4 rows for each of 64 experts of 4096 x 1408: 129 us, with
    // 128-tiles 146 us; 256 experts of 7168 x 2048: 1.40 and 1.25 ms.  dx, 2 rows for each of 32
    // experts of 2048 x 2048: 61 and 42 us; 16 rows of one 4096 x 4096: 13 and 32 us.)
    plan.kernel = kStream;
    plan.split = parts(red / 1024, 256 / stream);
    if (plan.split < 3 && mode == kLinear) plan.split = 1;  // the joining launch costs as much
  } else if (rows > 448 && n256 >= 256) {
    // (406 rows per expert, 4096 -> 1408: 458 us with 128-tiles, 498 us with 256-tiles; 512
    // rows, 7168 -> 2048: 5.2 ms and 4.0 ms)
    plan.kernel = kTile256;
  } else if (n128 >= 384) {
    // (4000 x 2048 x 2048: 41 us, 52 us with 64-tiles; 1003 x 1416 x 2056, 136 tiles: 26 us and
    // 22 us)
    // (4 rows for each of 256 experts, 7168 -> 2048: 1289 us, with the non-temporal hint 1167 us;
    // 100 rows for each of 128, 2048 -> 768: 116 us and 107 us)
    plan.kernel = rows <= 96 ? kTile128Once : kTile128;
  } else {
    // few tiles: long reductions in parts (100 x 7168 x 1024: 36 -> 16 us; 153 tiles of
    // 1034 x 4096 x 1056: 38 us, 28 in 2 parts, 24 in 3; of 1034 x 1416 x 1056: 16 us, 18 in 2)
    plan.split = parts(red / 1000, 512 / n64);
  }
  if (plan.split > 1)
    plan.ws_bytes = align256((size_t)plan.split * 4 *
                             (mode == kDw ? (size_t)p.E * (p.K + 1) * p.N  // and dbias's
                                           : (size_t)p.R * ncols));
  return plan;
}

hipError_t launch_grouped_linear(const moe_grouped& p, const void* x, const int32_t* row_token,
                                 const int32_t* offsets, const void* w, const void* bias, int act,
                                 const void* residual, void* y, uint8_t* codes, uint8_t* scales,
                                 void* ws, hipStream_t s) {
  GroupedArgs g{(const uint16_t*)x, (const uint16_t*)w, row_token, offsets, (const uint16_t*)bias,
                (const uint16_t*)residual, (uint16_t*)y, nullptr, codes, scales, nullptr, nullptr,
                p.R, p.T, p.K, p.N, p.E, act, 0, 1, nullptr};
  return run_grouped(p, g, kLinear, ws, s);
}

hipError_t launch_grouped_dx(const moe_grouped& p, const void* dz, const int32_t* offsets,
                             const void* w, int act, const uint8_t* codes, const uint8_t* scales,
                             void* dx, void* a, void* ws, hipStream_t s) {
  GroupedArgs g{(const uint16_t*)dz, (const uint16_t*)w, nullptr, offsets, nullptr, nullptr,
                (uint16_t*)dx, (uint16_t*)a, const_cast<uint8_t*>(codes),
                const_cast<uint8_t*>(scales), nullptr, nullptr, p.R, p.T, p.K, p.N, p.E, act, 0, 1,
                nullptr};
  return run_grouped(p, g, kDx, ws, s);
}

hipError_t launch_grouped_dw(const moe_grouped& p, const void* x, const int32_t* row_token,
                             const void* dz, const int32_t* offsets, int accumulate, float* dw,
                             float* dbias, void* ws, hipStream_t s) {
  if (p.R == 0) row_token = nullptr;  // no rows: only zeros to store, no list to read
  GroupedArgs g{(const uint16_t*)x, (const uint16_t*)dz, row_token, offsets, nullptr, nullptr,
                nullptr, nullptr, nullptr, nullptr, dw, dbias, p.R, p.T, p.K, p.N, p.E, 0,
                accumulate, 1, nullptr};
  return run_grouped(p, g, kDw, ws, s);
}

size_t grouped_ws_bytes(const moe_grouped& p, int op) { return grouped_plan(p, op).ws_bytes; }

hipError_t launch_act_backward(int64_t rows, int cols, const int32_t* live, int act,
                               const void* dy, const uint8_t* codes, const uint8_t* scales,
                               void* dz, void* a, hipStream_t s) {
  // a launch holds fewer than 2^32 threads: 2^32 values at a time
  constexpr int64_t kBlocks = 1 << 21;
  static_assert(kBlocks * 256 < (int64_t)1 << 32, "");
  const int64_t n8 = rows * (cols / 8);
  for (int64_t at = 0; at < n8; at += kBlocks * 256) {
    const int64_t blocks = std::min(div_up64(n8 - at, 256), kBlocks);
    hipLaunchKernelGGL(act_backward_kernel, dim3((unsigned)blocks), dim3(256), 0, s, at, n8,
                       cols / 8, live, act, (const uint4*)dy, (const uint2*)codes, scales,
                       (uint4*)dz, (uint4*)a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
