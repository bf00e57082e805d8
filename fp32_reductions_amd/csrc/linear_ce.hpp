// linear_ce.hpp -- host-side interface between the C ABI (api.hip) and the
// kernels of the output layer's cross entropy (linear_ce.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.hpp"
#include "rowloss.hpp"

namespace red {

// Rows, vocabulary, width and row strides, so that tile numbers and the byte
// offsets within a tile fit 32 bits.
constexpr size_t kLinearRowsMax = size_t(1) << 20;
constexpr size_t kLinearVocabMax = size_t(1) << 24;
constexpr size_t kLinearWidthMax = size_t(1) << 16;
constexpr size_t kLinearStrideMax = size_t(1) << 21;

struct LinearCall {
    const void *hidden, *weight;
    size_t rows, D, ldh, V, ldw;
    const int64_t* targets;
    const float* row_weight;
    float scale, z;
    float *loss, *logp, *lse;
    int accum;
    void *dhidden, *dweight;
    size_t lddh, lddw;
    void* workspace;
    size_t workspace_bytes;
};

// Bytes of workspace that the call needs (its pointers only say which outputs
// are wanted); the sizes within the limits above all fit size_t.
size_t linear_ce_workspace(const LinearCall& a, const DeviceInfo& dev);
hipError_t launch_linear_ce(LogitType t, const LinearCall& a, const DeviceInfo& dev,
                            hipStream_t stream);

} // namespace red
