// Launchers of the grouped linear products (natural weight layout); the arguments are those of
// the C entries.  Apart from moe_internal.h: the layer's kernels do not depend on them, and their
// sources keep the state that the recorded memory traffic was measured on.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

#ifdef MOE_DEBUG_CHECKS
// ---- dispatch.hip: offsets (if not NULL) non-decreasing inside [0, R], row_token (if not NULL)
// of the rows they name inside [0, T).
hipError_t launch_check_grouped(const moe_grouped& g, const int32_t* offsets,
                                const int32_t* row_token, hipStream_t s);
#endif

// ---- grouped.hip
hipError_t launch_grouped_linear(const moe_grouped& g, const void* x, const int32_t* row_token,
                                 const int32_t* offsets, const void* w, const void* bias, int act,
                                 const void* residual, void* y, uint8_t* codes, uint8_t* scales,
                                 void* ws, hipStream_t s);
hipError_t launch_grouped_dx(const moe_grouped& g, const void* dz, const int32_t* offsets,
                             const void* w, int act, const uint8_t* codes, const uint8_t* scales,
                             void* dx, void* a, void* ws, hipStream_t s);
hipError_t launch_grouped_dw(const moe_grouped& g, const void* x, const int32_t* row_token,
                             const void* dz, const int32_t* offsets, int accumulate, float* dw,
                             float* dbias, void* ws, hipStream_t s);
// Workspace of a moe_grouped_op.
size_t grouped_ws_bytes(const moe_grouped& g, int op);
hipError_t launch_act_backward(int64_t rows, int cols, const int32_t* live, int act,
                               const void* dy, const uint8_t* codes, const uint8_t* scales,
                               void* dz, void* a, hipStream_t s);

}  // namespace moe
