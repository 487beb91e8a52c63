// Launchers of the mixture-of-experts operators (not installed).  Arguments are already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tq2_moe.h"

namespace tq2 {

// Parts of the hidden axis whose sums the choice joins.
int route_parts(int64_t tokens, int64_t experts, int64_t hidden);
hipError_t launch_moe_route(const tq2_moe_route_args& a, hipStream_t stream);

// Layout of a call of tq2_moe_experts.
struct MoePlan {
  size_t y_offset;           // of the weighted rows in the workspace, behind the rows between the projections
  size_t items_offset;       // of the pairs sorted by expert
  size_t workspace;
};
MoePlan plan_moe(const tq2_moe_experts_args& a);
hipError_t launch_moe_experts(const tq2_moe_experts_args& a, const MoePlan& plan, hipStream_t stream);

}  // namespace tq2
