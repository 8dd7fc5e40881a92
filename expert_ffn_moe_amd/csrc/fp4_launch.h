// Launchers of the 4-bit forms (quant_fp4.hip) and of the grouped product on them
// (grouped_fp4.hip); the arguments are those of the C entries.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// ---- quant_fp4.hip
hipError_t launch_quantize_fp4(const void* x, int64_t rows, int cols, const int32_t* live,
                               uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_quantize_fp4_weights(const void* w, int E, int K, int N, uint8_t* codes,
                                       uint8_t* scales, hipStream_t s);
hipError_t launch_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                 int cols, const int32_t* live, void* out, hipStream_t s);

// ---- grouped_fp4.hip
using Fp4Weights = moe_fp4_weights;
hipError_t launch_grouped_fp4(const moe_grouped& g, bool eight, const uint8_t* x_codes,
                              const uint8_t* x_scales, const int32_t* row_token,
                              const int32_t* offsets, const Fp4Weights& w, const Fp4Weights& up,
                              int act, const void* residual, void* y, void* ws, hipStream_t s);
size_t grouped_fp4_ws_bytes(const moe_grouped& g);

}  // namespace moe
