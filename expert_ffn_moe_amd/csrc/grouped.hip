// Grouped linear products with their epilogues and gradients (moe_grouped_linear, _dx, _dw,
// moe_activation_backward): bf16 operands from their natural layouts, fp32 accumulation.
//
// LightLLM PR #1687 (PR body): the expert GEMMs run on the expert prefix-sum layout; the row
// count of every expert is data dependent and is read on the device from `offsets`.
//
//   linear  z = x W + b,  y = act(z) + residual, z kept as E4M3 codes with UE8M0 scales
//   dx      dx = (dz W^T) act'(z),  a = act(z)
//   dw      dW = x^T dz,  db = sum of dz
#include <algorithm>

#include "act.h"
#include "bf16.h"
#include "grouped_tile.h"
#include "moe_internal.h"
#include "wave.h"

namespace moe {
namespace {

constexpr int kXcds = 8;

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

// One output tile.
struct Item {
  int e;      // expert
  int m0;     // linear, dx: first row; dw: first of K
  int rows;   // live rows of the tile
  int n0;     // first output column
  int lo;     // dw: first row of the reduction
  int red;    // length of the reduction
};

// Persistent: the blocks of an XCD (workgroups go to XCDs round-robin) take the items of its
// contiguous share in turn, expert by expert, the M tiles of an N group next to each other, so
// that the operand bytes the items share come from that XCD's L2.  The next item's first
// stage is copied while the last one of the current item computes.
template <int MODE, bool GATHER, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2)))
void tile_kernel(const GroupedArgs g) {
  constexpr int NT = 64 * WM * WN;
  constexpr int FM = BM / 16 / WM, FN = BN / 16 / WN;  // fragments of a wavefront
  constexpr int AMODE = MODE == kDw ? kCols : kRows, BMODE = MODE == kDx ? kRows : kCols;
  using A = Operand<AMODE, BM, NT>;
  using B = Operand<BMODE, BN, NT>;
  constexpr int kSlot = A::kBytes + B::kBytes;
  __shared__ __align__(1024) char smem[2 * kSlot];
  __shared__ int s_start[kMaxE + 1];
  __shared__ int s_wsum[WM * WN];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(MOE_LDS char*)smem;
  const int ncols = MODE == kDx ? g.K : g.N;
  const int ntn = div_up(ncols, BN);

  // ---- the items of this block's XCD
  int lo_t, items;  // linear, dx: M tiles; dw: (expert, K tile) pairs
  const int xcd = blockIdx.x % kXcds, slots = gridDim.x / kXcds;
  {
    int total;
    if constexpr (MODE == kDw) {
      total = g.E * div_up(g.K, BM);
    } else {
      const int per = div_up(g.E, NT);
      const int e0 = min(g.E, tid * per), e1 = min(g.E, e0 + per);
      int sum = 0, lo, hi;
      for (int e = e0; e < e1; ++e) {
        segment(g.offsets, g.R, e, lo, hi);
        sum += div_up(hi - lo, BM);
      }
      const int inc = wave_inclusive_scan(sum);
      if (lane == 63) s_wsum[wave] = inc;
      __syncthreads();
      int base = inc - sum;
      for (int w = 0; w < wave; ++w) base += s_wsum[w];
      for (int e = e0; e < e1; ++e) {
        segment(g.offsets, g.R, e, lo, hi);
        s_start[e] = base;
        base += div_up(hi - lo, BM);
      }
      if (tid == NT - 1) s_start[g.E] = base;
      __syncthreads();
      total = s_start[g.E];
    }
    lo_t = (int)((int64_t)total * xcd / kXcds);
    items = ((int)((int64_t)total * (xcd + 1) / kXcds) - lo_t) * ntn;
  }
  auto find = [&](int item) {
    Item t;
    if constexpr (MODE == kDw) {
      const int ntk = div_up(g.K, BM), q = lo_t + item / ntn;
      t.e = q / ntk;
      t.m0 = (q - t.e * ntk) * BM;
      t.rows = min(BM, g.K - t.m0);
      t.n0 = (item % ntn) * BN;
      int hi;
      segment(g.offsets, g.R, t.e, t.lo, hi);
      t.red = hi - t.lo;
    } else {
      const int hi_t = lo_t + items / ntn;
      int lo = 0, hi = g.E;
      const int q = lo_t + item / ntn;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= q) lo = mid; else hi = mid;
      }
      t.e = __builtin_amdgcn_readfirstlane(lo);
      // the expert's items in this share: N group major, M tile minor
      const int seg0 = max(s_start[t.e], lo_t), nte = min(s_start[t.e + 1], hi_t) - seg0;
      const int local = item - ntn * (seg0 - lo_t);
      const int nt = local / nte, mt = seg0 + (local - nt * nte) - s_start[t.e];
      int beg, end;
      segment(g.offsets, g.R, t.e, beg, end);
      t.m0 = __builtin_amdgcn_readfirstlane(beg + mt * BM);
      t.rows = __builtin_amdgcn_readfirstlane(min(BM, end - t.m0));
      t.n0 = __builtin_amdgcn_readfirstlane(nt * BN);
      t.lo = 0;
      t.red = MODE == kLinear ? g.K : g.N;
    }
    return t;
  };

  // ---- copies: each piece is base + 32-bit offset, the base moving on by a stage; gathered
  // rows have an address of their own (linear) or are looked up stage by stage (dw)
  uint32_t a_off[A::kLoads], b_off[B::kLoads];
  const char *a_base, *b_base;
  const char* a_ptr[MODE == kLinear && GATHER ? A::kLoads : 1];
  int tok[MODE == kDw && GATHER ? A::kLoads : 1];  // rows of the next stage to be copied
  int tok_row = 0, tok_left = 0;
  const char* const zeros = reinterpret_cast<const char*>(g_zeros);
  const size_t a_ld = 2 * (size_t)(MODE == kDx ? g.N : g.K);  // bytes of a row of A
  const size_t b_ld = 2 * (size_t)g.N;
  const size_t a_step = AMODE == kRows ? 2 * kStage : kStage * a_ld;
  const size_t b_step = BMODE == kRows ? 2 * kStage : kStage * b_ld;
  auto load_tokens = [&]() {
#pragma unroll
    for (int i = 0; i < A::kLoads; ++i) {
      const int r = A::row_of(tid, i);
      tok[i] = r < tok_left ? g.row_token[tok_row + r] : 0;
    }
  };
  auto setup = [&](const Item& t, int tid) {
    a_base = (const char*)g.x + (AMODE == kRows ? (GATHER ? 0 : t.m0 * a_ld)
                                                : (GATHER ? 0 : t.lo * a_ld) + 2 * (size_t)t.m0);
    b_base = (const char*)g.w + (MODE == kLinear ? (size_t)t.e * g.K * b_ld + 2 * (size_t)t.n0
                                 : MODE == kDx   ? ((size_t)t.e * g.K + t.n0) * b_ld
                                                 : t.lo * b_ld + 2 * (size_t)t.n0);
#pragma unroll
    for (int i = 0; i < A::kLoads; ++i) {
      const int r = A::row_of(tid, i), c = A::piece_of(tid, i) * 8;
      if constexpr (AMODE == kRows) {  // rows behind the tile's last repeat it
        const int row = min(r, t.rows - 1);
        if constexpr (GATHER) {
          // a token outside x reads row 0 here and zeros in the epilogue
          const int tk = g.row_token[t.m0 + row];
          a_ptr[i] = a_base + ((unsigned)tk < (unsigned)g.T ? tk : 0) * a_ld + 2 * c;
        } else {
          a_off[i] = (uint32_t)(row * a_ld) + 2 * c;
        }
      } else {  // columns behind the last repeat it
        const int col = min(c, g.K - 8 - t.m0);
        a_off[i] = (GATHER ? 0 : (uint32_t)(r * a_ld)) + 2 * col;
      }
    }
#pragma unroll
    for (int i = 0; i < B::kLoads; ++i) {
      const int r = B::row_of(tid, i), c = B::piece_of(tid, i) * 8;
      b_off[i] = BMODE == kRows ? (uint32_t)(min(r, ncols - 1 - t.n0) * b_ld) + 2 * c
                                : (uint32_t)(r * b_ld) + 2 * min(c, ncols - 8 - t.n0);
    }
    if constexpr (MODE == kDw && GATHER) {
      tok_row = t.lo;
      tok_left = t.red;
      load_tokens();
    }
  };
  // One stage into a slot; left: what remains of the reduction (less than a stage: the rest of
  // both operands reads as zeros).
  auto issue = [&](int slot, int left, int rows) {
    const uint32_t la = __builtin_amdgcn_readfirstlane(lds0 + slot * kSlot + wave * 1024);
    const uint32_t lb = la + A::kBytes;
#pragma unroll
    for (int i = 0; i < A::kLoads; ++i) {
      // rows behind the tile's last: their fragments are garbage and not stored
      if (AMODE == kRows && i * A::kRowsPerLoad >= rows) break;
      if (!GATHER && left >= kStage) {
        copy_to_lds(a_base, a_off[i], la + i * NT * 16);
      } else {
        const char* src;
        if constexpr (MODE == kLinear && GATHER)
          src = a_ptr[i];
        else if constexpr (MODE == kDw && GATHER)
          src = (unsigned)tok[i] < (unsigned)g.T ? a_base + tok[i] * a_ld + a_off[i] : zeros;
        else
          src = a_base + a_off[i];
        if (left < kStage) {
          const int at = AMODE == kRows ? A::piece_of(tid, i) * 8 : A::row_of(tid, i);
          src = at < left ? src : zeros;
        }
        copy_to_lds(src, la + i * NT * 16);
      }
      if constexpr (MODE == kLinear && GATHER) a_ptr[i] += a_step;
    }
#pragma unroll
    for (int i = 0; i < B::kLoads; ++i) {
      if (left >= kStage) {
        copy_to_lds(b_base, b_off[i], lb + i * NT * 16);
      } else {
        const int at = BMODE == kRows ? B::piece_of(tid, i) * 8 : B::row_of(tid, i);
        copy_to_lds(at < left ? b_base + b_off[i] : zeros, lb + i * NT * 16);
      }
    }
    if (!GATHER) a_base += a_step;
    b_base += b_step;
    if constexpr (MODE == kDw && GATHER) {
      tok_row += kStage;
      tok_left -= kStage;
      load_tokens();
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
  auto compute = [&](int slot, auto nm_c) {
    constexpr int NM = decltype(nm_c)::value;
    if constexpr (NM == 0) return;
    const uint32_t so = slot * kSlot;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      bf16x8_t av[NM > 0 ? NM : 1], bv[FN];
#pragma unroll
      for (int n = 0; n < FN; ++n)
        bv[n] = BMODE == kRows ? read_rows(fb[kk] + so + n * 2048)
                               : read_cols<BN>(fb[n] + so + kk * 64 * BN);
#pragma unroll
      for (int m = 0; m < NM; ++m)
        av[m] = AMODE == kRows ? read_rows(fa[kk] + so + m * WM * 2048)
                               : read_cols<BM>(fa[m] + so + kk * 64 * BM);
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[n], av[m], acc[m][n], 0, 0, 0);
    }
  };

  // ---- epilogue: the columns are the instruction's rows, so a lane holds 4 consecutive
  // columns n0 + wcol + 16 n + 4 (lane / 16) .. + 3 of row lane % 16 of each fragment.
  auto epilogue = [&](const Item& t, int nm) {
    // through an empty statement: otherwise what derives from the lane below is computed
    // before the items' loop and kept in registers through it
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int c4 = t.n0 + wcol + 4 * (lane >> 4);
    if constexpr (MODE == kDw) {
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const int r = (m * WM + wm) * 16 + (lane & 15);
        if (r >= t.rows) continue;
        float* o = g.dw + ((size_t)t.e * g.K + t.m0 + r) * g.N + c4;
#pragma unroll
        for (int n = 0; n < FN; ++n) {
          if (c4 + 16 * n >= g.N) continue;
          f32x4_t v = acc[m][n];
          if (g.accumulate) v += *(const f32x4_t*)(o + 16 * n);
          *(f32x4_t*)(o + 16 * n) = v;
        }
      }
    } else {
      static_assert(FN % 2 == 0, "pairs of fragments");
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
        if (m >= nm) break;  // wave-uniform
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
      }
    }
  };

  int idx = blockIdx.x / kXcds;
  if (idx >= items) return;  // block-uniform
  Item cur = find(idx), nxt = cur;
  setup(cur, tid);
  issue(0, cur.red, cur.rows);
  wait_copies();
  int slot = 0;
  for (;;) {
    const int nst = max(1, div_up(cur.red, kStage));
    // fragments of this wavefront with live rows; none where all its columns are outside
    const int nm = cur.n0 + wcol >= ncols ? 0 : min(FM, div_up(cur.rows - wm * 16, 16 * WM));
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int n = 0; n < FN; ++n) acc[m][n] = f32x4_t{};
    auto stages = [&](auto nm_c) {  // all but the last
      for (int s = 0; s < nst - 1; ++s) {
        if (s > 0) wait_copies();
        block_barrier();
        issue(slot ^ 1, cur.red - (s + 1) * kStage, cur.rows);
        compute(slot, nm_c);
        slot ^= 1;
      }
    };
    constexpr int kHalf = FM / 2, kQuarter = FM >= 4 ? FM / 4 : 1;
    if (nm > kHalf)
      stages(std::integral_constant<int, FM>{});
    else if (nm > kQuarter)
      stages(std::integral_constant<int, kHalf>{});
    else if (nm > 0)
      stages(std::integral_constant<int, kQuarter>{});
    else
      stages(std::integral_constant<int, 0>{});
    if (nst > 1) wait_copies();
    block_barrier();
    idx += slots;
    const bool more = idx < items;
    if (more) {
      int tid_v = tid;  // as in the epilogue
      asm volatile("" : "+v"(tid_v));
      nxt = find(idx);
      setup(nxt, tid_v);
      issue(slot ^ 1, nxt.red, nxt.rows);
    }
    if (nm > kHalf)
      compute(slot, std::integral_constant<int, FM>{});
    else if (nm > kQuarter)
      compute(slot, std::integral_constant<int, kHalf>{});
    else if (nm > 0)
      compute(slot, std::integral_constant<int, kQuarter>{});
    slot ^= 1;
    wait_copies();  // the next item's first stage, before the stores join the count
    if (nm > 0) epilogue(cur, nm);
    if (!more) return;
    cur = nxt;
  }
}

// db[e][n]: a block per expert and 64 columns; 32 row lanes of 8 threads (8 columns each) take
// the rows in turn and are added up in order.
__global__ __launch_bounds__(256) void dbias_kernel(const GroupedArgs g) {
  __shared__ float part[32][64 + 1];
  const int e = blockIdx.y, c = threadIdx.x % 8 * 8, rl = threadIdx.x / 8;
  const int n = blockIdx.x * 64 + c;
  int lo, hi;
  segment(g.offsets, g.R, e, lo, hi);
  float s[8] = {};
  if (n < g.N)
    for (int r = lo + rl; r < hi; r += 32) {
      float f[8];
      unpack8(*(const uint4*)(g.w + (size_t)r * g.N + n), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += f[i];
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[rl][c + i] = s[i];
  __syncthreads();
  const int col = blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x >= 64 || col >= g.N) return;
  float v = 0.0f;
  for (int r = 0; r < 32; ++r) v += part[r][threadIdx.x];
  float* d = g.dbias + (size_t)e * g.N + col;
  *d = g.accumulate ? *d + v : v;
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
void launch_tiles(const GroupedArgs& g, hipStream_t s) {
  const int rows = MODE == kDw ? g.K : g.R / g.E;
  if (rows > 160)
    hipLaunchKernelGGL((tile_kernel<MODE, GATHER, 256, 256, 2, 4>), dim3(cu_count()), dim3(512), 0,
                       s, g);
  else
    hipLaunchKernelGGL((tile_kernel<MODE, GATHER, 128, 128, 2, 2>), dim3(2 * cu_count()),
                       dim3(256), 0, s, g);
}

}  // namespace

hipError_t launch_grouped_linear(const moe_grouped& p, const void* x, const int32_t* row_token,
                                 const int32_t* offsets, const void* w, const void* bias, int act,
                                 const void* residual, void* y, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s) {
  GroupedArgs g{(const uint16_t*)x, (const uint16_t*)w, row_token, offsets, (const uint16_t*)bias,
                (const uint16_t*)residual, (uint16_t*)y, nullptr, codes, scales, nullptr, nullptr,
                p.R, p.T, p.K, p.N, p.E, act, 0};
  if (row_token)
    launch_tiles<kLinear, true>(g, s);
  else
    launch_tiles<kLinear, false>(g, s);
  return hipGetLastError();
}

hipError_t launch_grouped_dx(const moe_grouped& p, const void* dz, const int32_t* offsets,
                             const void* w, int act, const uint8_t* codes, const uint8_t* scales,
                             void* dx, void* a, hipStream_t s) {
  GroupedArgs g{(const uint16_t*)dz, (const uint16_t*)w, nullptr, offsets, nullptr, nullptr,
                (uint16_t*)dx, (uint16_t*)a, const_cast<uint8_t*>(codes),
                const_cast<uint8_t*>(scales), nullptr, nullptr, p.R, p.T, p.K, p.N, p.E, act, 0};
  launch_tiles<kDx, false>(g, s);
  return hipGetLastError();
}

hipError_t launch_grouped_dw(const moe_grouped& p, const void* x, const int32_t* row_token,
                             const void* dz, const int32_t* offsets, int accumulate, float* dw,
                             float* dbias, hipStream_t s) {
  GroupedArgs g{(const uint16_t*)x, (const uint16_t*)dz, row_token, offsets, nullptr, nullptr,
                nullptr, nullptr, nullptr, nullptr, dw, dbias, p.R, p.T, p.K, p.N, p.E, 0,
                accumulate};
  if (row_token)
    launch_tiles<kDw, true>(g, s);
  else
    launch_tiles<kDw, false>(g, s);
  if (dbias)
    hipLaunchKernelGGL(dbias_kernel, dim3(div_up(p.N, 64), p.E), dim3(256), 0, s, g);
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
