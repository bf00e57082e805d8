// rowloss_join.hpp -- where the row losses (or pair losses) of a launch meet.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "rowloss.hpp"

namespace red {

// Each row's loss goes to the workspace, and the wave whose row is the last
// to arrive adds them up, in the order of the rows.  A second kernel for the
// sum took 3.2 us more of host time a call and 1.4 us and a gap on the GPU
// (96 rows of 32768 bf16: 15.6 us a call against 10.6).  A row's loss is stored, has arrived where every compute die sees it
// (a device-scope store, waited for), and only then is the row counted, so
// the last one finds all.  A release fence would do as well, but would write
// back the whole L2 with the gradient in it.  The last wave sets the count
// back to zero for the next launch on the stream.  Past kJoinRows rows, whose
// sum is too much for one wave, `count` is null and a kernel of its own
// adds them up.
constexpr uint32_t kJoinRows = 1024;
struct Join {
    double* row_loss;
    unsigned* count;
    float* loss;
    int accum;
    __device__ __forceinline__ void put(size_t row, double v) const
    {
        __hip_atomic_store(reinterpret_cast<unsigned long long*>(row_loss + row),
                           __builtin_bit_cast(unsigned long long, v), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
    // By every lane of the wave whose lane 0 has put the row's loss.
    __device__ __forceinline__ unsigned arrive() const
    {
        unsigned before = 0;
        if (count && (threadIdx.x & 63) == 0) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        return before;
    }
    // By the same wave with what arrive() gave lane 0.
    __device__ __forceinline__ void finish(unsigned before, uint32_t rows) const
    {
        if (!count || __builtin_amdgcn_readfirstlane(before) != rows - 1)
            return;
        const uint32_t lane = threadIdx.x & 63;
        const float old = accum ? loss[0] : 0.0f;
        double sum = 0.0;
        for (uint32_t i = lane; i < rows; i += 8 * kWave) {
            unsigned long long v[8];
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k)
                v[k] = i + k * kWave < rows
                           ? __hip_atomic_load(reinterpret_cast<unsigned long long*>(row_loss) + i +
                                                   k * kWave,
                                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                           : 0ull;
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k)
                sum += __builtin_bit_cast(double, v[k]);
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1)
            sum += __shfl_xor(sum, m);
        if (lane == 0) {
            loss[0] = (float)((double)old + sum);
            __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
};

// For operators without a loss to join.
struct NoJoin {
    __device__ __forceinline__ unsigned arrive() const { return 0; }
    __device__ __forceinline__ void finish(unsigned, uint32_t) const {}
};

// The meeting place of `rows` losses at `row_loss` (in the workspace).
inline Join join_of(const Workspace& ws, void* row_loss, size_t rows, float* loss, int accum)
{
    return {static_cast<double*>(row_loss), rows <= kJoinRows ? ws.counter : nullptr, loss, accum};
}

// After the launch that puts them: the sum, where no wave of it adds them up.
inline hipError_t sum_joined(const Join& j, size_t rows, hipStream_t stream)
{
    return j.count ? hipSuccess : launch_loss_sum(j.row_loss, rows, j.loss, j.accum, stream);
}

} // namespace red
