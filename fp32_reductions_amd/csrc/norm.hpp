// norm.hpp -- host-side interface between the C ABI (api.hip) and the kernels
// of the root-mean-square norm (norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.hpp"
#include "rowloss.hpp"

namespace red {

// Columns of a row, which stays in the registers of one workgroup.
constexpr size_t kNormColsMax = 16384;

struct NormCall {
    const void *x, *residual, *weight;
    void *sum, *y;
    uint8_t* y8;
    float *scale8, *rstd;
    size_t rows, D, ldx, ldr, lds, ldy, ldy8;
    float eps;
};

struct NormGradCall {
    const void *h, *weight;
    const float* rstd;
    const void *dy, *dsum;
    void* dx;
    float* dweight;
    size_t rows, D, ldh, lddy, ldds, lddx;
    int accum;
};

hipError_t launch_add_rmsnorm(LogitType t, const NormCall& a, const DeviceInfo& dev,
                              hipStream_t stream);
hipError_t launch_rmsnorm_grad(LogitType t, const NormGradCall& a, const DeviceInfo& dev,
                               const Workspace& ws, hipStream_t stream);

} // namespace red
