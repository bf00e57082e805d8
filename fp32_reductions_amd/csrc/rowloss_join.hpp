// rowloss_join.hpp -- where the row losses (or pair losses) of a launch meet.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "rowloss.hpp"

namespace red {

// Each row's loss goes to the workspace, and the wave whose row is the last
// to arrive adds them up, in a fixed order.  A second kernel for the sum took
// 3.2 us more of host time a call and 1.4 us and a gap on the GPU (96 rows of
// 32768 bf16: 15.6 us a call against 10.6).  A row's loss is stored, has
// arrived where every compute die sees it (a device-scope store, waited for),
// and only then is the row counted, so the last one finds all.  A release
// fence would do as well, but would write back the whole L2 with the gradient
// in it.  This is gfx950's behaviour and not the language's memory model, by
// which relaxed stores and a relaxed count order nothing: device-scope stores
// write through to where every die reads, s_waitcnt vmcnt(0) returns once they
// have, device-scope loads do not read an older copy, and they are issued after
// a branch on the count that was returned.  Another target needs the fences.
//
// Arrivals at one address follow each other at 12 ns (1024 rows of 1000 bf16:
// 17.1 us with one count, 4.3 us for one row), so every 64 rows have a count
// of their own, on its own cache lines; the last of 64 adds up their losses
// and arrives with the sum at the next level.  The last ones set the counts
// back to zero for the next launch on the stream.  Past kJoinRows rows
// `count` is null and a kernel of its own adds up.
constexpr uint32_t kJoinGroup = kWave, kJoinGroups = 256;
constexpr uint32_t kJoinRows = kJoinGroup * kJoinGroups;
constexpr uint32_t kCountStride = 64; // words between counts

// Sum over a wave in fp64, in every lane: by DPP as in wave_reduce, a lane's
// two halves at a time.  (With __shfl_xor, an LDS permute for each half and
// step, a sum took three times as long: distillation of 1 row of 1000 with 32
// entries and the rest 6.0 us a call, 5.6 so.)  All lanes take part.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_add64(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)b, CTRL, ROW_MASK, 0xf, false);
    const unsigned hi =
        __builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), CTRL, ROW_MASK, 0xf, false);
    return v + __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}

__device__ __forceinline__ double wave_sum64(double v)
{
    v = dpp_add64<0x111, 0xf>(v); // row_shr:1
    v = dpp_add64<0x112, 0xf>(v); // row_shr:2
    v = dpp_add64<0x114, 0xf>(v); // row_shr:4
    v = dpp_add64<0x118, 0xf>(v); // row_shr:8
    v = dpp_add64<0x142, 0xa>(v); // row_bcast:15 -> rows 1, 3
    v = dpp_add64<0x143, 0xc>(v); // row_bcast:31 -> rows 2, 3
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = __builtin_amdgcn_readlane((int)(unsigned)b, 63);
    const unsigned hi = __builtin_amdgcn_readlane((int)(unsigned)(b >> 32), 63);
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}

// Words that workgroups on different compute dies share within a launch.
__device__ __forceinline__ void store_shared(double* p, double v)
{
    __hip_atomic_store(reinterpret_cast<unsigned long long*>(p),
                       __builtin_bit_cast(unsigned long long, v), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_shared(float* p, float v)
{
    __hip_atomic_store(reinterpret_cast<unsigned*>(p), __float_as_uint(v), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double load_shared(const double* p)
{
    return __builtin_bit_cast(
        double, __hip_atomic_load(reinterpret_cast<const unsigned long long*>(p), __ATOMIC_RELAXED,
                                  __HIP_MEMORY_SCOPE_AGENT));
}
__device__ __forceinline__ float load_shared(const float* p)
{
    return __uint_as_float(__hip_atomic_load(reinterpret_cast<const unsigned*>(p),
                                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}
// One more arrival, after everything this lane has stored; the count before.
__device__ __forceinline__ unsigned count_shared(unsigned* p)
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    return __hip_atomic_fetch_add(p, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void clear_shared(unsigned* p)
{
    __hip_atomic_store(p, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

struct Join {
    double* row_loss;
    double* group_sum;
    unsigned* count; // [0]: of groups; [1 + g]: of the rows of group g
    float* loss;
    int accum;
    __device__ __forceinline__ void put(size_t row, double v) const { store_shared(row_loss + row, v); }
    // By every lane of the wave whose lane 0 has put the row's loss.
    __device__ __forceinline__ unsigned arrive(uint32_t row) const
    {
        return count ? arrive_at(count + (1 + row / kJoinGroup) * kCountStride) : 0;
    }
    // By the same wave with what arrive() gave lane 0.
    __device__ __forceinline__ void finish(unsigned before, uint32_t row, uint32_t rows) const
    {
        if (!count)
            return;
        const uint32_t lane = threadIdx.x & 63, g = row / kJoinGroup;
        const uint32_t first = g * kJoinGroup;
        const uint32_t size = rows - first < kJoinGroup ? rows - first : kJoinGroup;
        if (__builtin_amdgcn_readfirstlane(before) != size - 1)
            return;
        double sum = wave_sum64(lane < size ? load_shared(row_loss + first + lane) : 0.0);
        if (lane == 0)
            clear_shared(count + (1 + g) * kCountStride);
        const uint32_t groups = (rows + kJoinGroup - 1) / kJoinGroup;
        if (groups > 1) {
            if (lane == 0)
                store_shared(group_sum + g, sum);
            before = arrive_at(count);
            if (__builtin_amdgcn_readfirstlane(before) != groups - 1)
                return;
            double v[kJoinGroups / kWave];
#pragma unroll
            for (uint32_t k = 0; k < kJoinGroups / kWave; ++k)
                v[k] = lane + k * kWave < groups ? load_shared(group_sum + lane + k * kWave) : 0.0;
            sum = 0.0;
#pragma unroll
            for (uint32_t k = 0; k < kJoinGroups / kWave; ++k)
                sum += v[k];
            sum = wave_sum64(sum);
            if (lane == 0)
                clear_shared(count);
        }
        if (lane == 0)
            loss[0] = (float)((accum ? (double)loss[0] : 0.0) + sum);
    }

  private:
    static __device__ __forceinline__ unsigned arrive_at(unsigned* p)
    {
        return (threadIdx.x & 63) == 0 ? count_shared(p) : 0;
    }
};
static_assert((1 + kJoinGroups) * kCountStride <= kCounterWords, "a count for each group");
static_assert(kJoinRows < kRowsPerLaunch, "a loss of several launches has no count");

// For operators without a loss to join.
struct NoJoin {
    __device__ __forceinline__ unsigned arrive(uint32_t) const { return 0; }
    __device__ __forceinline__ void finish(unsigned, uint32_t, uint32_t) const {}
};

// The meeting place of `rows` losses at `row_loss` (in the workspace).  A loss of
// several launches has no count (its rows are more than kJoinRows): its sum
// passes from one to the next in fp64, in the word before the groups' sums.
inline Join join_of(const Workspace& ws, void* row_loss, size_t rows, float* loss, int accum)
{
    return {static_cast<double*>(row_loss),
            reinterpret_cast<double*>(static_cast<char*>(ws.partials) + ws.partial_bytes) -
                kJoinGroups,
            rows <= kJoinRows ? ws.counters : nullptr, loss, accum};
}

// After the launch that puts them: the sum, where no wave of it adds them up.
// first, last: of the launches that make the loss.
inline hipError_t sum_joined(const Join& j, size_t rows, hipStream_t stream, bool first = true,
                             bool last = true)
{
    double* passed = j.group_sum - 1;
    return j.count ? hipSuccess
                   : launch_loss_sum(j.row_loss, rows, j.loss, j.accum, first ? nullptr : passed,
                                     last ? nullptr : passed, stream);
}

} // namespace red
