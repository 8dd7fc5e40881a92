// Routing by scores: softmax or sigmoid scores of the router's logits, experts chosen by
// score + bias under a group limit, weights from the scores alone (LightLLM PR #1687,
// call-order paragraph: the layer's `experts()` does grouped top-k and renormalises).
//
//   score   s = 1 / (1 + exp(-l)), or exp(l - m) / sum exp(l - m)
//   order   s + b, or the logits themselves without a bias (the scores rise with them)
//   weight  c s / (sum of the chosen s), or c s
//
// Choices are made and weights computed in 64 bits and each weight is rounded once: a choice
// next to a border, and the capacity's comparison of weights, do then not depend on how an
// exponential was rounded to 32 bits.
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
  double scale;
};

constexpr float kBig = 3.402823466e38f;

// Order-preserving map of fp64 (with -0 folded into +0) to uint64; every number maps above 1.
__device__ __forceinline__ uint64_t ordered_bits(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v == 0.0 ? 0.0 : v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}

// NaN and -inf, as a logit or a bias: the expert is out; +inf counts as the largest number.
__device__ __forceinline__ bool is_in(float v) { return v > -INFINITY; }

// One wavefront per token; a lane holds experts lane, lane + 64, ...
template <int EPL>  // E <= 64 * EPL
__global__ __launch_bounds__(256) void scored_kernel(const ScoredArgs a) {
  __shared__ double s_val[4][64 * EPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wave;
  if (t >= a.T) return;  // wave-uniform
  const float* row = a.logits + (size_t)t * a.E;
  float l[EPL];
  bool in[EPL], can[EPL];  // part of the softmax; to be chosen
  double c[EPL];           // what the experts are ordered by
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    float v = -INFINITY;
    if (e < a.E) {
      v = row[e];
#pragma unroll 8
      for (int q = 1; q < a.S; ++q) v = v + row[q * a.plane + e];
      if (a.logits_out) a.logits_out[(size_t)t * a.E + e] = v;
    }
    in[i] = is_in(v);
    can[i] = in[i] && (!a.bias || is_in(a.bias[e]));
    l[i] = fminf(v, kBig);
    c[i] = l[i];
  }
  const bool grouped = a.n_group > 1 && a.topk_group < a.n_group;
  const bool by_score = grouped && a.group_score == MOE_GROUP_TOP2;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  float m = 0.0f;
  double total = 1.0;  // of the softmax over all experts
  if (softmax) {
    m = -kBig;
#pragma unroll
    for (int i = 0; i < EPL; ++i) m = in[i] ? fmaxf(m, l[i]) : m;
    m = wave_max(m);
  }
  auto score_of = [&](float v) {
    return softmax ? exp((double)v - (double)m) : 1.0 / (1.0 + exp(-(double)v));
  };
  double s[EPL];
  const bool all = a.bias || by_score || (softmax && !a.renorm);
  if (all) {
    total = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = in[i] ? score_of(l[i]) : 0.0;
      total += s[i];
    }
    total = softmax ? wave_sum(total) : 1.0;
    if (!(total > 0.0)) total = 1.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] /= total;
      if (a.bias && lane + 64 * i < a.E) {
        s[i] += (double)fminf(a.bias[lane + 64 * i], kBig);
        c[i] = s[i];
      }
    }
  }
  // 0: not to be chosen, 1: out (chosen last, lowest id first), else the order
  uint64_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    key[i] = lane + 64 * i >= a.E ? 0 : can[i] ? ordered_bits(c[i]) : 1;
  if (grouped) {
    const int gs = a.E / a.n_group;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      s_val[wave][lane + 64 * i] = can[i] ? (by_score ? s[i] : c[i]) : -INFINITY;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // this wavefront's own values
    __builtin_amdgcn_wave_barrier();
    uint64_t g = 0;
    if (lane < a.n_group) {
      double v1 = -INFINITY, v2 = -INFINITY;
      for (int q = 0; q < gs; ++q) {
        const double v = s_val[wave][lane * gs + q];
        v2 = fmax(v2, fmin(v1, v));
        v1 = fmax(v1, v);
      }
      if (by_score && v2 > -INFINITY) v1 += v2;
      g = ordered_bits(v1);
    }
    int ahead = 0;
    for (int q = 0; q < a.n_group; ++q) {
      const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)g, q);
      const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(g >> 32), q);
      const uint64_t o = ((uint64_t)hi << 32) | lo;
      ahead += o > g || (o == g && q < lane);
    }
    const uint64_t taken = __ballot(lane < a.n_group && ahead < a.topk_group);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 64 * i < a.E && !((taken >> ((lane + 64 * i) / gs)) & 1)) key[i] = 0;
  }
  // k rounds of a maximum; equal keys: the lowest expert
  int my_e = 0;
  float my_l = 0.0f;
  bool my_in = false;
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = max_u64(best, key[i]);
    best = wave_max_u64(best);
    int e = 0;
    float v = 0.0f;
    bool found = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint64_t at = __ballot(key[i] == best);
      if (!found && at) {  // wave-uniform
        const int src = __builtin_ctzll(at);
        e = src + 64 * i;
        v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(l[i]), src));
        if (lane == src) key[i] = 0;
        found = true;
      }
    }
    if (lane == j) {
      my_e = e;
      my_l = v;
      my_in = best > 1;
    }
  }
  double w = lane < a.k && my_in ? score_of(my_l) / total : 0.0;
  if (a.renorm) {
    const double sum = wave_sum(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < a.k) {
    const size_t o = (size_t)t * a.k + lane;
    a.ids[o] = my_e;
    a.w[o] = (float)(a.scale * w);
    a.keep[o] = my_in;
  }
}

struct ScoredBwdArgs {
  const float* logits;
  const int32_t* ids;
  const float* w;
  const float* dw;
  float* dl;
  int T, E, k, renorm, score;
};

// The gradient of the logits from that of the weights (the choice itself carries none), with
// d_j the gradient of slot j, w_j its weight (0 where the expert was out), p the softmax:
//   sigmoid, renormalised  dl_j = w_j (1 - s_j) (d_j - D),  D = sum w d / sum w
//   sigmoid                dl_j = w_j (1 - s_j) d_j
//   softmax, renormalised  dl_j = w_j (d_j - D)
//   softmax                dl_e = [e chosen] w_e d_e - p_e sum w d
// In 64 bits, for d_j - D cancels.  One wavefront per token.
template <int EPL>
__global__ __launch_bounds__(256) void scored_bwd_kernel(const ScoredBwdArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.T) return;  // wave-uniform
  const float* row = a.logits + (size_t)t * a.E;
  const size_t o = (size_t)t * a.k;
  const bool mine = lane < a.k;
  const int e = mine ? a.ids[o + lane] : -1;
  const double w = mine ? (double)a.w[o + lane] : 0.0;
  const double d = mine && w != 0.0 ? (double)a.dw[o + lane] : 0.0;
  double D = wave_sum(w * d);
  double g = w * d;
  if (a.renorm) {
    const double sum = wave_sum(w);
    D = sum != 0.0 ? D / sum : 0.0;
    g = w * (d - D);
  }
  if (a.score == MOE_SCORE_SIGMOID && w != 0.0 && (unsigned)e < (unsigned)a.E)
    g /= 1.0 + exp((double)fminf(row[e], kBig));
  double p[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) p[i] = 0.0;
  if (a.score == MOE_SCORE_SOFTMAX && !a.renorm) {
    float l[EPL];
    float m = -kBig;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int q = lane + 64 * i;
      l[i] = q < a.E ? row[q] : -INFINITY;
      m = is_in(l[i]) ? fmaxf(m, fminf(l[i], kBig)) : m;
    }
    m = wave_max(m);
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = is_in(l[i]) ? exp((double)fminf(l[i], kBig) - (double)m) : 0.0;
      total += p[i];
    }
    total = wave_sum(total);
    const double f = total > 0.0 ? -D / total : 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] *= f;
  }
  for (int j = 0; j < a.k; ++j) {
    const int ej = __builtin_amdgcn_readlane(e, j);
    const double gj = __shfl(g, j, 64);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 64 * i == ej) p[i] += gj;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (lane + 64 * i < a.E) a.dl[(size_t)t * a.E + lane + 64 * i] = (float)p[i];
}

}  // namespace

hipError_t launch_route_scored(const moe_problem& p, const moe_scoring& sc, const float* logits,
                               int S, const float* bias, float* logits_out, int32_t* ids, float* w,
                               uint8_t* keep, hipStream_t s) {
  const ScoredArgs a{logits, bias, logits_out, ids, w, keep, (size_t)p.T * p.E, S, p.T, p.E, p.k,
                     p.renormalize, sc.score, sc.n_group, sc.topk_group, sc.group_score, sc.scale};
  const dim3 grid(div_up(p.T, 4)), block(256);
  if (p.E <= 64) hipLaunchKernelGGL(scored_kernel<1>, grid, block, 0, s, a);
  else if (p.E <= 128) hipLaunchKernelGGL(scored_kernel<2>, grid, block, 0, s, a);
  else if (p.E <= 256) hipLaunchKernelGGL(scored_kernel<4>, grid, block, 0, s, a);
  else if (p.E <= 512) hipLaunchKernelGGL(scored_kernel<8>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(scored_kernel<16>, grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(const moe_problem& p, const moe_scoring& sc,
                                   const float* logits, const int32_t* ids, const float* w,
                                   const float* dw, float* dlogits, hipStream_t s) {
  const ScoredBwdArgs a{logits, ids, w, dw, dlogits, p.T, p.E, p.k, p.renormalize, sc.score};
  const dim3 grid(div_up(p.T, 4)), block(256);
  if (p.E <= 64) hipLaunchKernelGGL(scored_bwd_kernel<1>, grid, block, 0, s, a);
  else if (p.E <= 128) hipLaunchKernelGGL(scored_bwd_kernel<2>, grid, block, 0, s, a);
  else if (p.E <= 256) hipLaunchKernelGGL(scored_bwd_kernel<4>, grid, block, 0, s, a);
  else if (p.E <= 512) hipLaunchKernelGGL(scored_bwd_kernel<8>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(scored_bwd_kernel<16>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
