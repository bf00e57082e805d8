// rowloss.hip -- what the losses over rows of logits share whatever the
// element type: the sum of row losses, the pairs of a preference loss, and
// the choice of the element type.
//
// Everything here is a few numbers per row or pair, in fp64 and in a fixed
// order: a sum of thousands of row losses of both signs keeps its last fp32
// bits and is the same in every run.
#include "device.hpp"
#include "rowloss.hpp"
#include "rowloss_pairs.hpp"

namespace red {
namespace {

// Sum over a workgroup of WAVES waves, in every thread.  lds: WAVES doubles,
// free when the call begins.
template <int WAVES>
__device__ __forceinline__ double block_sum64(double v, double* lds)
{
    v = wave_sum64(v);
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x / 64] = v;
    __syncthreads();
    double s = lds[0];
#pragma unroll
    for (int k = 1; k < WAVES; ++k)
        s += lds[k];
    return s;
}

// One workgroup: thread t adds terms t, t + 1024, ..., four loads in flight.
__global__ __launch_bounds__(1024) void loss_sum_kernel(const double* __restrict__ v, uint32_t n,
                                                        float* loss, int accum,
                                                        const double* before, double* after)
{
    __shared__ double lds[16];
    const double old = before ? before[0] : accum ? (double)loss[0] : 0.0;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (uint32_t i = threadIdx.x; i < n; i += 4096) {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
            s[k] += i + k * 1024 < n ? v[i + k * 1024] : 0.0;
    }
    const double sum = block_sum64<16>((s[0] + s[1]) + (s[2] + s[3]), lds);
    if (threadIdx.x != 0)
        return;
    if (after)
        after[0] = old + sum;
    else
        loss[0] = (float)(old + sum);
}

// One workgroup per pair.  Sequence p is the chosen one and P + p the
// rejected; bounds outside [0, rows] are moved into it.
__global__ __launch_bounds__(256) void preference_pairs_kernel(PairArgs a)
{
    __shared__ double lds[4][4];
    const uint32_t p = blockIdx.x;
    const PairValues values(a, p);
    int64_t begin[2], end[2];
    double sum[2], count[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const uint64_t i = (uint64_t)side * a.pairs + p;
        int64_t b = a.starts[i], e = a.starts[i + 1];
        b = b < 0 ? 0 : b > a.rows ? a.rows : b;
        e = e < b ? b : e > a.rows ? a.rows : e;
        double s = 0.0, n = 0.0;
        for (int64_t r = b + threadIdx.x; r < e; r += 256) {
            s += load_shared(a.row_logp + r); // 0 where the target is not a column
            n += (uint64_t)a.targets[r] < (uint64_t)a.V ? 1.0 : 0.0;
        }
        begin[side] = b;
        end[side] = e;
        sum[side] = block_sum64<4>(s, lds[2 * side]);
        count[side] = block_sum64<4>(n, lds[2 * side + 1]);
    }
    const PairResult pair(a, values, sum, count);
    if (threadIdx.x == 0)
        pair.put(a, p);
    const unsigned before = threadIdx.x < kWave ? a.join.arrive(p) : 0;
#pragma unroll
    for (int side = 0; side < 2; ++side)
        for (int64_t r = begin[side] + threadIdx.x; r < end[side]; r += 256)
            a.row_slope[r] = pair.slope[side];
    if (threadIdx.x < kWave)
        a.join.finish(before, p, a.pairs);
}

} // namespace

hipError_t launch_loss_sum(const double* row_loss, size_t n, float* loss, int accum,
                           const double* before, double* after, hipStream_t stream)
{
    hipLaunchKernelGGL(loss_sum_kernel, dim3(1), dim3(1024), 0, stream, row_loss, (uint32_t)n,
                       loss, accum, before, after);
    return hipGetLastError();
}

hipError_t launch_preference_pairs(const PairArgs& args, hipStream_t stream)
{
    hipLaunchKernelGGL(preference_pairs_kernel, dim3(args.pairs), dim3(256), 0, stream, args);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? sum_joined(args.join, args.pairs, stream) : e;
}

#define RED_BY_TYPE(t, call)                        \
    switch (t) {                                    \
    case LogitType::F32: return RowLoss<ElemF32>::call; \
    case LogitType::F16: return RowLoss<ElemF16>::call; \
    default: return RowLoss<ElemBF16>::call;        \
    }

bool token_logprob_shares(LogitType t, const Logits& m) { RED_BY_TYPE(t, logprob_shares(m)) }
hipError_t launch_token_logprob(LogitType t, const LogprobCall& a, const DeviceInfo& dev,
                                const Workspace& ws, hipStream_t stream)
{
    RED_BY_TYPE(t, logprob(a, dev, ws, stream))
}
hipError_t launch_token_logprob_grad(LogitType t, const LogprobGradCall& a,
                                     const DeviceInfo& dev, hipStream_t stream)
{
    RED_BY_TYPE(t, logprob_grad(a, dev, stream))
}
hipError_t launch_distill_topk(LogitType t, const DistillCall& a, const DeviceInfo& dev,
                               const Workspace& ws, hipStream_t stream)
{
    RED_BY_TYPE(t, distill(a, dev, ws, stream))
}
hipError_t launch_policy_loss(LogitType t, const PolicyCall& a, const DeviceInfo& dev,
                              const Workspace& ws, hipStream_t stream)
{
    RED_BY_TYPE(t, policy(a, dev, ws, stream))
}
hipError_t launch_preference_loss(LogitType t, const PreferenceCall& a, const DeviceInfo& dev,
                                  const Workspace& ws, hipStream_t stream)
{
    RED_BY_TYPE(t, preference(a, dev, ws, stream))
}

} // namespace red
