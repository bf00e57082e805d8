// router.hpp -- host-side interface between the C ABI (api.hip) and the kernels
// of a router's balance loss (router.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.hpp"
#include "rowloss.hpp"

namespace red {

// Experts of a router: a wave holds a row, and each workgroup's counts are in LDS.
constexpr size_t kRouterExpertsMax = 2048;

struct RouterCall {
    Logits m; // V: experts
    const int64_t* experts;
    size_t K, ldk;
    const float* weight;
    float balance, z;
    float* loss;
    int64_t* counts;
    float* prob;
    int accum;
};

hipError_t launch_router_balance(LogitType t, const RouterCall& a, const DeviceInfo& dev,
                                 const Workspace& ws, hipStream_t stream);

} // namespace red
