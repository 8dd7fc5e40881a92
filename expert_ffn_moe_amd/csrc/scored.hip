// Routing by scores: softmax or sigmoid scores of the router's logits, experts chosen by
// score + bias under a group limit, weights from the scores alone (LightLLM PR #1687,
// call-order paragraph: the layer's `experts()` does grouped top-k and renormalises).
//
//   score   s = 1 / (1 + exp(-l)), or exp(l - m) / sum exp(l - m)
//   order   s + b, or the logits themselves without a bias (the scores rise with them)
//   weight  c s / (sum of the chosen s), or c s
//
// Choices are those of 64-bit scores and weights are computed in 64 bits and rounded once: a
// choice next to a border, and the capacity's comparison of weights, do then not depend on how an
// exponential was rounded to 32 bits.  Most choices are nowhere near a border: with up to 256
// experts, 8 choices and groups of whole lanes a token is first taken in 32 bits, and again in 64
// only where two of the values that decided lay closer than their error bounds (or were equal, or
// an expert that is out would be needed).  All others are taken in 64 bits alone.
#include <algorithm>
#include <initializer_list>

#include "moe_internal.h"
#include "scored.h"
#include "wave.h"

namespace moe {
namespace {

struct ScoredArgs {
  const float* logits;  // S planes [T, E], added in order
  const float* bias;
  float* logits_out;
  int32_t* ids;
  float* w;
  uint8_t* keep;
  size_t plane;
  int S, T, E, k, renorm, score, n_group, topk_group, group_score;
  int vec;   // rows can be read in words of min(EPL, 4) values
  int span;  // rows kernel under a group limit: the lanes of a group, 1, 2, 4 or 8
  double scale;
};

constexpr float kBig = 3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;

// Order-preserving map of fp64 (with -0 folded into +0) to uint64; every number maps above 1.
__device__ __forceinline__ uint64_t ordered_bits(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v == 0.0 ? 0.0 : v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

constexpr int kDppRowNext = 0x101;  // row_shl:1: the next lane of the row (0 behind the last)

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v)));
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
// Over the 16 lanes of a row, the same in each.
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_f<kDppQuadXor1>(v);
  v += dpp_f<kDppQuadXor2>(v);
  v += dpp_f<kDppRowHalfMirror>(v);
  return v + dpp_f<kDppRowMirror>(v);
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  return __builtin_bit_cast(double, dpp_u64<CTRL>(__builtin_bit_cast(uint64_t, v)));
}
__device__ __forceinline__ double row_sum(double v) {
  v += dpp_d<kDppQuadXor1>(v);
  v += dpp_d<kDppQuadXor2>(v);
  v += dpp_d<kDppRowHalfMirror>(v);
  return v + dpp_d<kDppRowMirror>(v);
}
__device__ __forceinline__ float from_lane(float v, int src) {
  return __uint_as_float(__builtin_amdgcn_ds_bpermute(4 * src, (int)__float_as_uint(v)));
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp_f<kDppQuadXor1>(v));
  v = fmaxf(v, dpp_f<kDppQuadXor2>(v));
  v = fmaxf(v, dpp_f<kDppRowHalfMirror>(v));
  return fmaxf(v, dpp_f<kDppRowMirror>(v));
}
__device__ __forceinline__ uint32_t row_top(uint32_t v) {
  v = max(v, dpp_u32<kDppQuadXor1>(v));
  v = max(v, dpp_u32<kDppQuadXor2>(v));
  v = max(v, dpp_u32<kDppRowHalfMirror>(v));
  return max(v, dpp_u32<kDppRowMirror>(v));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_f<kDppQuadXor1>(v));
  v = fmaxf(v, dpp_f<kDppQuadXor2>(v));
  v = fmaxf(v, dpp_f<kDppRowHalfMirror>(v));
  v = fmaxf(v, dpp_f<kDppRowMirror>(v));
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
// Order-preserving map of fp32 to uint32 and back.
__device__ __forceinline__ uint32_t ordered32(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered32(uint32_t o) {
  return __uint_as_float(o ^ ((uint32_t)(~(int32_t)o >> 31) | 0x80000000u));
}
constexpr uint32_t kOutKey = 0x007FFFFFu;  // of -inf

// exp(x) for x <= 0 in 64 bits: x = n ln 2 + r, |r| <= ln 2 / 2, the Taylor series of exp(r) to
// r^13 (the next term is below 2^-57 of it), times 2^n.
__device__ __forceinline__ double exp64(double x) {
  x = fmax(x, -1000.0);  // 0 from there on; -inf
  const double n = rint(x * 1.4426950408889634);
  // ln 2 as 0x1.62e42fee p-1 (n times it is exact) and the rest
  double r = fma(n, -0x1.62e42feep-1, x);
  r = fma(n, -0x1.a39ef35793c76p-33, r);
  double q = 1.0 / 6227020800.0;
  q = fma(q, r, 1.0 / 479001600.0);
  q = fma(q, r, 1.0 / 39916800.0);
  q = fma(q, r, 1.0 / 3628800.0);
  q = fma(q, r, 1.0 / 362880.0);
  q = fma(q, r, 1.0 / 40320.0);
  q = fma(q, r, 1.0 / 5040.0);
  q = fma(q, r, 1.0 / 720.0);
  q = fma(q, r, 1.0 / 120.0);
  q = fma(q, r, 1.0 / 24.0);
  q = fma(q, r, 1.0 / 6.0);
  q = fma(q, r, 0.5);
  q = fma(q, r, 1.0);
  q = fma(q, r, 1.0);
  return ldexp(q, (int)n);
}
// 1 / (1 + exp(-x))
__device__ __forceinline__ double sigmoid64(double x) {
  const double e = exp64(-fabs(x));
  return (x >= 0.0 ? 1.0 : e) / (1.0 + e);
}

// NaN and -inf, as a logit or a bias: the expert is out; +inf counts as the largest number.
__device__ __forceinline__ bool is_in(float v) { return v > -INFINITY; }
__device__ __forceinline__ float tamed(float v) { return is_in(v) ? fminf(v, kBig) : -INFINITY; }

// Values EPL lane .. EPL lane + EPL - 1 of a row of E; fill behind its end.
template <int EPL>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, bool vec, float fill,
                                         float (&v)[EPL]) {
  constexpr int W = EPL < 4 ? EPL : 4;
  typedef float word __attribute__((ext_vector_type(W)));
  if (vec) {  // uniform
#pragma unroll
    for (int i = 0; i < EPL; i += W) {
      word q;
#pragma unroll
      for (int j = 0; j < W; ++j) q[j] = fill;
      if (lane * EPL + i < E) q = *(const word*)(row + lane * EPL + i);
#pragma unroll
      for (int j = 0; j < W; ++j) v[i + j] = q[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = lane * EPL + i < E ? row[lane * EPL + i] : fill;
  }
}

// The logits of token t, planes added in order.
template <int EPL>
__device__ __forceinline__ void load_logits(const ScoredArgs& a, int t, int lane, float (&l)[EPL]) {
  const float* row = a.logits + (size_t)t * a.E;
  load_row<EPL>(row, a.E, lane, a.vec, -INFINITY, l);
  for (int p = 1; p < a.S; ++p) {
    float v[EPL];
    load_row<EPL>(row + p * a.plane, a.E, lane, a.vec, 0.0f, v);
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] += v[i];
  }
}

// The two largest of the disjoint sets of two lanes.
__device__ __forceinline__ void merge2(float& a1, float& a2, float b1, float b2) {
  a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
  a1 = fmaxf(a1, b1);
}

// The k choices of token t in 64 bits by one wavefront, a lane holding EPL consecutive experts:
// lane j returns the expert of slot j.  s_val: 64 EPL values of this wavefront's own.
template <int EPL>
__device__ __forceinline__ int choose64(const ScoredArgs& a, int t, int lane, double* s_val) {
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  const bool grouped = a.n_group > 1 && a.topk_group < a.n_group;
  const bool top2 = grouped && a.group_score == MOE_GROUP_TOP2;
  float l[EPL], b[EPL];
  load_logits<EPL>(a, t, lane, l);
#pragma unroll
  for (int i = 0; i < EPL; ++i) b[i] = 0.0f;
  if (a.bias) load_row<EPL>(a.bias, a.E, lane, a.vec, -INFINITY, b);
  float m = -kBig;
  double total = 0.0, d[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    l[i] = tamed(l[i]);
    b[i] = tamed(b[i]);
    m = fmaxf(m, l[i]);
    d[i] = 0.0;
  }
  m = wave_max(m);
  if (a.bias || top2) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      d[i] = !is_in(l[i]) ? 0.0
             : softmax    ? exp64((double)l[i] - (double)m)
                          : sigmoid64(l[i]);
      total += d[i];
    }
    total = softmax ? wave_sum(total) : 1.0;
    if (!(total > 0.0)) total = 1.0;
  }
  // 0: not to be chosen, 1: out (chosen last, lowest id first), else the order
  uint64_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const bool can = is_in(l[i]) && is_in(b[i]);
    if (a.bias || top2) d[i] = d[i] / total + (double)(can ? b[i] : 0.0f);
    const double by = a.bias ? d[i] : (double)l[i];
    key[i] = lane * EPL + i >= a.E ? 0 : can ? ordered_bits(by) : 1;
    if (grouped) s_val[lane * EPL + i] = can ? (top2 ? d[i] : by) : -INFINITY;
  }
  if (grouped) {
    const int gs = a.E / a.n_group;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // this wavefront's own values
    __builtin_amdgcn_wave_barrier();
    uint64_t g = 0;
    if (lane < a.n_group) {
      double v1 = -INFINITY, v2 = -INFINITY;
      for (int o = 0; o < gs; ++o) {
        const double v = s_val[lane * gs + o];
        v2 = fmax(v2, fmin(v1, v));
        v1 = fmax(v1, v);
      }
      if (top2 && v2 > -INFINITY) v1 += v2;
      g = ordered_bits(v1);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();  // before the next token's values
    int ahead = 0;
    for (int o = 0; o < a.n_group; ++o) {
      const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)g, o);
      const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(g >> 32), o);
      const uint64_t v = ((uint64_t)hi << 32) | lo;
      ahead += v > g || (v == g && o < lane);
    }
    const uint64_t taken = __ballot(lane < a.n_group && ahead < a.topk_group);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane * EPL + i < a.E && !((taken >> ((lane * EPL + i) / gs)) & 1)) key[i] = 0;
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = max_u64(best, key[i]);
    best = wave_max_u64(best);
    // equal keys: the lowest expert, in the lowest lane and there the lowest of its values
    uint64_t any = 0;
    int place = EPL;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i) {
      const bool hit = key[i] == best;
      any |= __ballot(hit);
      place = hit ? i : place;
    }
    const int src = __builtin_ctzll(any);
    const int at = __builtin_amdgcn_readlane(place, src);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane == src && i == at) key[i] = 0;
    mine = lane == j ? src * EPL + at : mine;
  }
  return mine;
}

// The weight of expert e of token t before scale and renormalisation, 0 where it is out (m, total:
// the softmax's), and whether it is in.
__device__ __forceinline__ double weight_of(const ScoredArgs& a, int t, int e, float m,
                                            double total, bool& in) {
  const float* at = a.logits + (size_t)t * a.E + e;
  float l = *at;
  for (int p = 1; p < a.S; ++p) l += at[p * a.plane];
  l = tamed(l);
  in = is_in(l) && (!a.bias || is_in(a.bias[e]));
  if (!in) return 0.0;
  return a.score == MOE_SCORE_SOFTMAX ? exp64((double)l - (double)m) / total : sigmoid64(l);
}

__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {  // the larger first
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
// Sorts 4 or 8 keys, largest first (odd-even merging).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t* v) {
  if constexpr (N == 4) {
    order2(v[0], v[1]); order2(v[2], v[3]);
    order2(v[0], v[2]); order2(v[1], v[3]);
    order2(v[1], v[2]);
  } else {
    sort_keys<4>(v);
    sort_keys<4>(v + 4);
    order2(v[0], v[4]); order2(v[1], v[5]); order2(v[2], v[6]); order2(v[3], v[7]);
    order2(v[2], v[4]); order2(v[3], v[5]);
    order2(v[1], v[2]); order2(v[3], v[4]); order2(v[5], v[6]);
  }
}

// A row of 16 lanes takes a token, a lane EPL consecutive experts: four tokens to a wavefront, every
// reduction inside a row.  Each lane sorts its keys first, so that a round of the choice is the
// maximum of the lanes' heads and the winner moves on to its next one.  For k <= 8 (a lane keeps 8
// keys) of up to 256 experts: 16384 tokens, 8 of 256 by groups, 16.5 to 17.5 us a call, where a
// wavefront for a token, in 64 bits throughout, took 38.6.  Its 16.8 MB are 3.7 us at the rate of a
// copy; the four wavefronts of a SIMD all load, then all compute (about 7 us of instructions), so
// that the two add up, with the launch's own start and end.
//
// In 32 bits a key is the order-preserving bits of the value, the last ones replaced by the value's
// place in its lane.  Bounds: a sigmoid from the hardware's exponential and reciprocal (1 ulp
// each) is off by at most 2^-22 (|l| s (1 - s) < 0.23 times the argument's rounding, 2^-24 for the
// sum, 2^-23 for the reciprocal), with the bias 2^-24 of the sum more; a softmax by at most 2^-19
// (its total by 25 2^-24 of itself).  Two values are told apart where they differ by more than
// the sum of their bounds, taken as eps (1 + |value|) with eps 2^-20 (2^-17 for the softmax) and
// EPL 2^-22 |value| for the keys.  A group's sum of two is held to its parts, for large biases
// may cancel in it: each is off by 2^-22 (1 + |part|) (2^-19 + 2^-24 |part|), the sum by 2^-24 of
// itself more, two groups by less than twice eps (1 + |part| + |part|) of the larger one together.
template <int EPL, bool SOFTMAX>  // E <= 16 * EPL
__global__ __launch_bounds__(256) void scored_rows_kernel(const ScoredArgs a) {
  constexpr int D = EPL < 8 ? EPL : 8;  // keys a lane keeps
  constexpr int kWide = EPL / 4;        // experts per lane where the wavefront takes one token
  __shared__ double s_val[4][64 * kWide];
  __shared__ int s_e[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15;
  const int t0 = (blockIdx.x * 4 + wave) * 4;
  if (t0 >= a.T) return;  // wave-uniform
  const int t = min(t0 + (lane >> 4), a.T - 1);
  const bool live = t0 + (lane >> 4) < a.T;
  const bool grouped = a.n_group > 1 && a.topk_group < a.n_group;
  const bool top2 = grouped && a.group_score == MOE_GROUP_TOP2;
  const bool scores = a.bias || top2;
  const float eps = SOFTMAX ? 0x1p-17f : 0x1p-20f;

  float l[EPL];
  load_logits<EPL>(a, t, l16, l);
  if (a.logits_out && live) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (l16 * EPL + i < a.E) a.logits_out[(size_t)t * a.E + l16 * EPL + i] = l[i];
  }
  float m = -kBig;
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] = tamed(l[i]);
  if constexpr (SOFTMAX) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) m = fmaxf(m, l[i]);
    m = row_max(m);
  }
  float s[EPL], c[EPL];  // the scores, and what the experts are ordered by
#pragma unroll
  for (int i = 0; i < EPL; ++i) s[i] = c[i] = l[i];
  if (scores) {
    float f = 1.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      s[i] = SOFTMAX ? __builtin_amdgcn_exp2f((l[i] - m) * kLog2e)
                     : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -kLog2e));
    if constexpr (SOFTMAX) {
      f = s[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) f += s[i];
      f = row_sum(f);
      f = f > 0.0f ? __builtin_amdgcn_rcpf(f) : 0.0f;
    }
    float b[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) b[i] = 0.0f;
    if (a.bias) load_row<EPL>(a.bias, a.E, l16, a.vec, -INFINITY, b);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      // (as a sum: for a choice between two values the compiler branches around the exponential)
      s[i] = fmaf(s[i], f, tamed(b[i])) + (is_in(l[i]) ? 0.0f : -INFINITY);
      c[i] = a.bias ? s[i] : c[i];
    }
  }
  bool unsure = false;
  if (grouped) {
    float v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float v = top2 ? s[i] : c[i];
      v2 = fmaxf(v2, fminf(v1, v));
      v1 = fmaxf(v1, v);
    }
    if (a.span > 1) merge2(v1, v2, dpp_f<kDppQuadXor1>(v1), dpp_f<kDppQuadXor1>(v2));
    if (a.span > 2) merge2(v1, v2, dpp_f<kDppQuadXor2>(v1), dpp_f<kDppQuadXor2>(v2));
    if (a.span > 4) merge2(v1, v2, dpp_f<kDppRowHalfMirror>(v1), dpp_f<kDppRowHalfMirror>(v2));
    const bool sum = top2 && is_in(v2);
    const float mine = sum ? v1 + v2 : v1;
    const float size = fabsf(v1) + (sum ? fabsf(v2) : 0.0f);
    // (ordered by the logits themselves only equal groups are close)
    const float near = scores ? 2.0f * eps * (1.0f + size) : 0.0f;
    int ahead = 0, close = 0;
    for (int o = 0; o < a.n_group; ++o) {
      const float v = from_lane(mine, (lane & 48) + o * a.span);
      ahead += v > mine;
      close += fabsf(v - mine) <= near;
    }
    // (each is close to itself; parts that pass the range together are left to 64 bits; a group that
    // is wholly out, -inf, is behind the others and close to none: with one group out 16384 tokens,
    // 8 of 256, took 54 us instead of 18 while it counted)
    unsure = ((close > 1 && is_in(v1)) || (sum && size > kBig)) && l16 < a.n_group * a.span;
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = ahead < a.topk_group ? c[i] : -INFINITY;
  }
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    key[i] = (ordered32(c[i]) & ~(uint32_t)(EPL - 1)) | (uint32_t)(EPL - 1 - i);
  if constexpr (EPL == 16) {  // the larger half, again in order
    sort_keys<8>(key);
    sort_keys<8>(key + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) key[i] = max(key[i], key[15 - i]);
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(i & d)) order2(key[i], key[i + d]);
  } else {
    sort_keys<EPL>(key);
  }
  uint32_t tops = 0, last = 0;  // lane j of a row: the key of round j; the first not chosen
  uint64_t twice = 0;           // rows in which two lanes had the same key
  for (int j = 0;; ++j) {
    last = row_top(key[0]);
    if (j == a.k) break;
    const bool win = key[0] == last;
    const uint64_t who = __ballot(win);
    twice |= who & (who - 0x0001000100010001ull);  // (each row has a winner)
    tops = l16 == j ? last : tops;
    if (win) s_e[wave][(lane & 48) + j] = l16 * EPL + (EPL - 1 - (int)(last & (EPL - 1)));
    // (as bits: the compiler made selects of the keys an indexed array, 190 instructions a round)
    const uint32_t next = win ? ~0u : 0u;
#pragma unroll
    for (int i = 0; i < D; ++i)
      key[i] = (next & (i + 1 < D ? key[i + 1] : 0)) | (~next & key[i]);
  }
  uint32_t after = dpp_u32<kDppRowNext>(tops);
  after = l16 == a.k - 1 ? last : after;
  const float v = unordered32(tops), w1 = unordered32(after);
  const float apart = (a.bias ? eps : 0x1p-126f) +
                      ((a.bias ? eps : 0.0f) + EPL * 0x1p-22f) * fmaxf(fabsf(v), fabsf(w1));
  // (out: fewer than k can be chosen; the first that is not chosen may be)
  unsure = unsure || (l16 < a.k && (tops <= kOutKey || (after > kOutKey && v - w1 <= apart))) ||
           (EPL > D && key[0] == 0);  // a lane whose next key is not known
  uint64_t again = (__ballot(unsure && live) | twice) & __ballot(live);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  int e = s_e[wave][lane];
  for (int r = 0; r < 4; ++r) {
    if (!((again >> (16 * r)) & 0xFFFF)) continue;  // wave-uniform
    int lane_v = lane;  // through an empty statement: nothing of this is computed ahead
    asm volatile("" : "+v"(lane_v));
    const int got = __shfl(choose64<kWide>(a, t0 + r, lane_v, s_val[wave]), lane & 15, 64);
    e = lane >> 4 == r ? got : e;
  }
  double total = 1.0;
  if (SOFTMAX && !a.renorm) {
    total = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) total += exp64((double)l[i] - (double)m);
    total = row_sum(total);
    if (!(total > 0.0)) total = 1.0;
  }
  bool in = false;
  double w = l16 < a.k ? weight_of(a, t, e, m, total, in) : 0.0;
  if (a.renorm) {
    const double sum = row_sum(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (live && l16 < a.k) {
    const size_t o = (size_t)t * a.k + l16;
    a.ids[o] = e;
    a.w[o] = (float)(a.scale * w);
    a.keep[o] = in;
  }
}

// A wavefront per token, for more experts or choices or groups that are not whole lanes; in 64 bits
// throughout, whose arithmetic and rounds of choice bound it.  16384 tokens with sigmoid scores and
// a bias: 8 of 384 48 us, 10 of 512 53, 8 of 512 in 8 groups 65, 16 of 256 43 (25, 34, 34 and 17 MB
// of logits are 5, 7, 7 and 3.5 us).
template <int EPL>  // E <= 64 * EPL
__global__ __launch_bounds__(256) void scored_wide_kernel(const ScoredArgs a) {
  __shared__ double s_val[4][64 * EPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wave;
  if (t >= a.T) return;  // wave-uniform
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  float m = 0.0f;
  double total = 1.0;
  if (softmax || a.logits_out) {
    float l[EPL];
    load_logits<EPL>(a, t, lane, l);
    m = -kBig;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (a.logits_out && lane * EPL + i < a.E)
        a.logits_out[(size_t)t * a.E + lane * EPL + i] = l[i];
      l[i] = tamed(l[i]);
      m = fmaxf(m, l[i]);
    }
    m = wave_max(m);
    if (softmax && !a.renorm) {
      total = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) total += exp64((double)l[i] - (double)m);
      total = wave_sum(total);
      if (!(total > 0.0)) total = 1.0;
    }
  }
  const int e = choose64<EPL>(a, t, lane, s_val[wave]);
  bool in = false;
  double w = lane < a.k ? weight_of(a, t, e, m, total, in) : 0.0;
  if (a.renorm) {
    const double sum = wave_sum(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < a.k) {
    const size_t o = (size_t)t * a.k + lane;
    a.ids[o] = e;
    a.w[o] = (float)(a.scale * w);
    a.keep[o] = in;
  }
}

struct ScoredBwdArgs {
  const float* logits;
  const int32_t* ids;
  const float* w;
  const float* dw;
  float* dl;
  int T, E, k, renorm, score, tokens, vec;
};

// The gradient of the logits from that of the weights (the choice itself carries none), with
// d_j the gradient of slot j, w_j its weight (0 where the expert was out), p the softmax:
//   sigmoid, renormalised  dl_j = w_j (1 - s_j) (d_j - D),  D = sum w d / sum w
//   sigmoid                dl_j = w_j (1 - s_j) d_j
//   softmax, renormalised  dl_j = w_j (d_j - D)
//   softmax                dl_e = [e chosen] w_e d_e - p_e sum w d
// In 64 bits, for d_j - D cancels.  A wavefront takes a.tokens tokens: their slots first, one to a
// lane, then their rows, a lane holding EPL consecutive experts.  Bound by the stores: 16384 x 256, 16.8
// MB of gradient, 9.1 us a call (softmax over all experts, which reads the logits too and takes
// their exponentials in 64 bits, 18 us).
template <int EPL>
__global__ __launch_bounds__(256) void scored_bwd_kernel(const ScoredBwdArgs a) {
  const int lane = threadIdx.x & 63;
  const int t0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * a.tokens;
  if (t0 >= a.T) return;  // wave-uniform
  const int nt = min(a.tokens, a.T - t0);
  const size_t o = (size_t)t0 * a.k + lane;
  const bool mine = lane < nt * a.k;
  const int e = mine ? a.ids[o] : -1;
  const double w = mine ? (double)a.w[o] : 0.0;
  const double d = w != 0.0 ? (double)a.dw[o] : 0.0;
  const int first = lane / a.k * a.k;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  double D = 0.0, sum = 0.0;
  if (a.renorm || softmax) {
    for (int j = 0; j < a.k; ++j) {
      D += __shfl(w * d, first + j, 64);
      sum += __shfl(w, first + j, 64);
    }
  }
  if (a.renorm) D = sum != 0.0 ? D / sum : 0.0;
  double g = w * (a.renorm ? d - D : d);
  // (+inf moves nothing: the sigmoid's slope is 0 there; beside it the softmax leaves weights to its
  // like alone, all equal, whose sum is exact, so that few tokens read their logits for it)
  const int n = __popcll(__ballot(w != 0.0) >> first & ((1ull << a.k) - 1));
  if (w != 0.0 && (!softmax || w * n == sum) && (unsigned)e < (unsigned)a.E) {
    const float l = a.logits[(size_t)(t0 + lane / a.k) * a.E + e];
    if (!softmax) g *= sigmoid64(-(double)fminf(l, kBig));
    else if (l == INFINITY) g = 0.0;
  }
  const float gf = (float)g;
  const bool dense = softmax && !a.renorm;
  for (int q = 0; q < nt; ++q) {
    const size_t row = (size_t)(t0 + q) * a.E;
    float v[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = 0.0f;
    if (dense) {
      double p[EPL];
      float l[EPL];
      load_row<EPL>(a.logits + row, a.E, lane, a.vec, -INFINITY, l);
      float m = -kBig;
      uint32_t moves = 0;  // values below +inf
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        moves |= (uint32_t)(l[i] < INFINITY) << i;
        l[i] = tamed(l[i]);
        m = fmaxf(m, l[i]);
      }
      m = wave_max(m);
      double total = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        p[i] = exp64((double)l[i] - (double)m);  // (out: -inf, or no expert at all)
        total += p[i];
      }
      total = wave_sum(total);
      const double f = total > 0.0 ? -__shfl(D, q * a.k, 64) / total : 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) p[i] *= f;
      for (int j = 0; j < a.k; ++j) {
        const int ej = __builtin_amdgcn_readlane(e, q * a.k + j);
        const double gj = __shfl(g, q * a.k + j, 64);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (lane * EPL + i == ej) p[i] += gj;
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = (moves >> i) & 1 ? (float)p[i] : 0.0f;
    } else {
      for (int j = 0; j < a.k; ++j) {
        const int ej = __builtin_amdgcn_readlane(e, q * a.k + j);
        const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gf), q * a.k + j));
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (lane * EPL + i == ej) v[i] += gj;
      }
    }
    constexpr int W = EPL < 4 ? EPL : 4;
    typedef float word __attribute__((ext_vector_type(W)));
    if (a.vec) {
#pragma unroll
      for (int i = 0; i < EPL; i += W) {
        word x;
#pragma unroll
        for (int j = 0; j < W; ++j) x[j] = v[i + j];
        // (written once: 16384 x 256 in 9.2 us with the hint, 10.7 without)
        if (lane * EPL + i < a.E)
          __builtin_nontemporal_store(x, (word*)(a.dl + row + lane * EPL + i));
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane * EPL + i < a.E) a.dl[row + lane * EPL + i] = v[i];
    }
  }
}

// Tokens per wavefront of the gradient: several share the pass over their slots where enough
// wavefronts remain (16384 tokens, before the stores had their hint: 10.7 us with 4, 12.7 with 1, 12.4
// with 8; 4096: 6.1 with 1, 7.6 with 2).
int tokens_per_wave(const moe_problem& p) {
  int n = 4;
  while (n > 1 && (n * p.k > 64 || p.T / n < 4096)) n /= 2;
  return n;
}
bool words_ok(int E, int epl, std::initializer_list<const void*> ptrs) {
  const int w = std::min(epl, 4);
  for (const void* q : ptrs)
    if ((uintptr_t)q % (4 * w) != 0) return false;
  return E % w == 0;
}
int experts_per_lane(int E) {
  int n = 1;
  while (64 * n < E) n *= 2;
  return n;
}

}  // namespace

#define MOE_BY_EPL(epl, kernel, ...)                                      \
  do {                                                                    \
    if ((epl) == 1) hipLaunchKernelGGL(kernel<1>, __VA_ARGS__);           \
    else if ((epl) == 2) hipLaunchKernelGGL(kernel<2>, __VA_ARGS__);      \
    else if ((epl) == 4) hipLaunchKernelGGL(kernel<4>, __VA_ARGS__);      \
    else if ((epl) == 8) hipLaunchKernelGGL(kernel<8>, __VA_ARGS__);      \
    else hipLaunchKernelGGL(kernel<16>, __VA_ARGS__);                     \
  } while (0)

hipError_t launch_route_scored(const moe_problem& p, const moe_scoring& sc, const float* logits,
                               int S, const float* bias, float* logits_out, int32_t* ids, float* w,
                               uint8_t* keep, hipStream_t s) {
  ScoredArgs a{logits, bias, logits_out, ids, w, keep, (size_t)p.T * p.E, S, p.T, p.E, p.k,
               p.renormalize, sc.score, sc.n_group, sc.topk_group, sc.group_score, 0, 0, sc.scale};
  const int lane_experts = p.E <= 64 ? 4 : p.E <= 128 ? 8 : 16, gs = p.E / sc.n_group;
  const int span = gs % lane_experts == 0 ? gs / lane_experts : 0;
  const bool lanes = span == 1 || span == 2 || span == 4 || span == 8;
  // Groups that are not whole lanes go to the other kernel: here they would all be chosen in 64 bits,
  // a token after the other (16384 tokens, 6 of 160 experts in 8 groups 43.6 us, there 35.2; 512
  // tokens 24.9 and 7.7; one 8.3 and 6.6; 4 of 72 in 8: 25.7 and 21.9, 15.7 and 5.6, 5.9 and 4.8).
  if (p.E <= 256 && p.k <= 8 && (lanes || sc.topk_group == sc.n_group)) {
    const int epl = lane_experts;
    // (the wavefront-wide form that the kernel falls back to reads smaller words of the same rows)
    a.vec = words_ok(p.E, 4, {logits, bias});
    a.span = span;
    const dim3 grid(div_up(p.T, 16)), block(256);
    const bool soft = sc.score == MOE_SCORE_SOFTMAX;
    if (epl == 4 && soft) hipLaunchKernelGGL((scored_rows_kernel<4, true>), grid, block, 0, s, a);
    else if (epl == 4) hipLaunchKernelGGL((scored_rows_kernel<4, false>), grid, block, 0, s, a);
    else if (epl == 8 && soft) hipLaunchKernelGGL((scored_rows_kernel<8, true>), grid, block, 0, s, a);
    else if (epl == 8) hipLaunchKernelGGL((scored_rows_kernel<8, false>), grid, block, 0, s, a);
    else if (soft) hipLaunchKernelGGL((scored_rows_kernel<16, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((scored_rows_kernel<16, false>), grid, block, 0, s, a);
  } else {
    const int epl = experts_per_lane(p.E);
    a.vec = words_ok(p.E, epl, {logits, bias});
    MOE_BY_EPL(epl, scored_wide_kernel, dim3(div_up(p.T, 4)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(const moe_problem& p, const moe_scoring& sc,
                                   const float* logits, const int32_t* ids, const float* w,
                                   const float* dw, float* dlogits, hipStream_t s) {
  const int epl = experts_per_lane(p.E);
  const ScoredBwdArgs a{logits, ids, w, dw, dlogits, p.T, p.E, p.k, p.renormalize, sc.score,
                        tokens_per_wave(p), words_ok(p.E, epl, {logits, dlogits})};
  MOE_BY_EPL(epl, scored_bwd_kernel, dim3(div_up(p.T, 4 * a.tokens)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
