// rowloss.hip -- what the losses over rows of logits share whatever the
// element type: the sum of row losses, the pairs of a preference loss, and
// the choice of the element type.
//
// Everything here is a few numbers per row or pair, in fp64 and in a fixed
// order: a sum of thousands of row losses of both signs keeps its last fp32
// bits and is the same in every run.
#include "device.hpp"
#include "reduce.h"
#include "rowloss.hpp"
#include "rowloss_join.hpp"

namespace red {
namespace {

// Sum over a workgroup of WAVES waves, in every thread.  lds: WAVES doubles,
// free when the call begins.
template <int WAVES>
__device__ __forceinline__ double block_sum64(double v, double* lds)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1)
        v += __shfl_xor(v, m);
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
                                                        float* loss, int accum)
{
    __shared__ double lds[16];
    const float old = accum ? loss[0] : 0.0f;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (uint32_t i = threadIdx.x; i < n; i += 4096) {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
            s[k] += i + k * 1024 < n ? v[i + k * 1024] : 0.0;
    }
    const double sum = block_sum64<16>((s[0] + s[1]) + (s[2] + s[3]), lds);
    if (threadIdx.x == 0)
        loss[0] = (float)((double)old + sum);
}

struct PairArgs {
    const double* row_logp;
    float* row_slope;
    const int64_t *targets, *starts;
    const float *ref_logp, *weight;
    float* seq_logp;
    Join join;
    int64_t rows, V;
    uint32_t pairs;
    int kind, average;
    double beta, margin, smoothing;
};

struct SequenceSum {
    int64_t begin, end;
    double logp, count;
};

// One workgroup per pair.  Sequence p is the chosen one and P + p the
// rejected; bounds outside [0, rows] are moved into it.
__global__ __launch_bounds__(256) void preference_pairs_kernel(PairArgs a)
{
    __shared__ double lds[4][4];
    const uint32_t p = blockIdx.x;
    SequenceSum seq[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const uint64_t i = (uint64_t)side * a.pairs + p;
        int64_t b = a.starts[i], e = a.starts[i + 1];
        b = b < 0 ? 0 : b > a.rows ? a.rows : b;
        e = e < b ? b : e > a.rows ? a.rows : e;
        double s = 0.0, n = 0.0;
        for (int64_t r = b + threadIdx.x; r < e; r += 256) {
            s += a.row_logp[r]; // 0 where the target is not a column
            n += (uint64_t)a.targets[r] < (uint64_t)a.V ? 1.0 : 0.0;
        }
        s = block_sum64<4>(s, lds[2 * side]);
        n = block_sum64<4>(n, lds[2 * side + 1]);
        seq[side] = {b, e, a.average && n > 0.0 ? s / n : s, a.average && n > 0.0 ? n : 1.0};
    }
    const double w = a.weight ? (double)a.weight[p] : 1.0 / (double)a.pairs;
    double delta = seq[0].logp - seq[1].logp;
    if (a.ref_logp)
        delta = (seq[0].logp - (double)a.ref_logp[p]) -
                (seq[1].logp - (double)a.ref_logp[(uint64_t)a.pairs + p]);
    const double h = a.beta * delta - a.margin;
    double loss, slope; // slope: d loss / d h
    if (a.kind == RED_PREF_SIGMOID) {
        // softplus(x) = max(x, 0) + log1p(exp(-|x|))
        const double t = exp(-fabs(h)), l = log1p(t);
        const double pos = fmax(h, 0.0) + l, neg = fmax(-h, 0.0) + l; // of h and of -h
        const double up = h >= 0.0 ? 1.0 / (1.0 + t) : t / (1.0 + t);  // sigmoid(h)
        const double down = h >= 0.0 ? t / (1.0 + t) : 1.0 / (1.0 + t);
        loss = (1.0 - a.smoothing) * neg + a.smoothing * pos;
        slope = a.smoothing * up - (1.0 - a.smoothing) * down;
    } else if (a.kind == RED_PREF_HINGE) {
        loss = h >= 1.0 ? 0.0 : 1.0 - h;
        slope = h >= 1.0 ? 0.0 : -1.0;
    } else {
        const double d = (h - 0.5) / a.beta;
        loss = d * d;
        slope = 2.0 * d / a.beta;
    }
    const double g = w != 0.0 ? w * slope * a.beta : 0.0;
    if (threadIdx.x == 0) {
        a.seq_logp[p] = (float)seq[0].logp;
        a.seq_logp[(uint64_t)a.pairs + p] = (float)seq[1].logp;
        a.join.put(p, w != 0.0 ? w * loss : 0.0);
    }
    const unsigned before = threadIdx.x < kWave ? a.join.arrive(p) : 0;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const float mine = (float)((side ? -g : g) / seq[side].count);
        for (int64_t r = seq[side].begin + threadIdx.x; r < seq[side].end; r += 256)
            a.row_slope[r] = mine;
    }
    if (threadIdx.x < kWave)
        a.join.finish(before, p, a.pairs);
}

} // namespace

hipError_t launch_loss_sum(const double* row_loss, size_t n, float* loss, int accum,
                           hipStream_t stream)
{
    hipLaunchKernelGGL(loss_sum_kernel, dim3(1), dim3(1024), 0, stream, row_loss, (uint32_t)n,
                       loss, accum);
    return hipGetLastError();
}

hipError_t launch_preference_pairs(const PreferenceCall& a, const double* row_logp,
                                   float* row_slope, const Join& join, hipStream_t stream)
{
    const PairArgs args = {row_logp,     row_slope,  a.targets,         a.starts,
                           a.ref_logp,   a.weight,   a.seq_logp,        join,
                           (int64_t)a.m.rows, (int64_t)a.m.V, (uint32_t)a.pairs, a.kind,
                           a.average,    a.beta,     a.margin,          a.smoothing};
    hipLaunchKernelGGL(preference_pairs_kernel, dim3((uint32_t)a.pairs), dim3(256), 0, stream,
                       args);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? sum_joined(join, a.pairs, stream) : e;
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
