// Launchers of the routing by scores; the arguments are those of the C entries.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// ---- route.hip
// The router's logits as router_plan's partial planes [split][T][E] in `part`.
hipError_t launch_router_logits(const moe_problem& p, const void* x, const void* wr, float* part,
                                hipStream_t s);

// ---- dispatch.hip
// Capacity over the slots themselves, for few tokens (no layout, no scratch).
bool capacity_direct(const moe_problem& p);
hipError_t launch_capacity_direct(const moe_problem& p, const int32_t* ids,
                                  const uint8_t* candidates, const float* topk_w, uint8_t* keep,
                                  hipStream_t s);

// ---- scored.hip
// Selection from S planes [T, E] of fp32 logits, added in plane order (S = 1: the logits); the
// sums are also written to logits_out if it is not NULL.
hipError_t launch_route_scored(const moe_problem& p, const moe_scoring& sc, const float* logits,
                               int S, const float* bias, float* logits_out, int32_t* ids, float* w,
                               uint8_t* keep, hipStream_t s);
hipError_t launch_route_scored_bwd(const moe_problem& p, const moe_scoring& sc,
                                   const float* logits, const int32_t* ids, const float* w,
                                   const float* dw, float* dlogits, hipStream_t s);

}  // namespace moe
