// Grouped products on microscaled operands (moe_grouped_linear_fp4): weights in 4 bits, x in 4 or
// 8, fp32 accumulation on the scaled matrix cores, epilogue as moe_grouped_linear.
//
// LightLLM PR #1687 (PR body): the expert GEMMs run on the expert prefix-sum layout with block
// scales that are powers of two.
#include "grouped_fp4.h"
#include "moe_internal.h"

namespace moe {

size_t grouped_fp4_ws_bytes(const moe_grouped&) { return 0; }

hipError_t launch_grouped_fp4(const moe_grouped& p, bool eight, const uint8_t* x_codes,
                              const uint8_t* x_scales, const int32_t* row_token,
                              const int32_t* offsets, const Fp4Weights& w, const Fp4Weights& up,
                              int act, const void* residual, void* y, void* ws, hipStream_t s) {
  const Fp4Args g{x_codes, x_scales, row_token, offsets, w, up, (const uint16_t*)residual,
                  (uint16_t*)y, p.R, p.T, p.K, p.N, p.E, act, 1, (float*)ws};
  return launch_fp4_stream(g, eight, s);
}

}  // namespace moe
