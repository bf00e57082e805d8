// router.hip -- the balance loss of a router of experts, its counts and its
// gradient.
//
//     p = softmax(z_r),  P_e = sum_r w_r p_re,  n_e: how often the rows that
//     count chose expert e,  f = n / sum n
//     loss = b E sum_e f_e P_e + c sum_r w_r lse_r^2
//     dz_r = w_r p_r (q - sum_e p_re q_e + 2 c lse_r),  q = b E f
//
// A row is short (its experts), and the rows are many: 4, 16 or 64 lanes share
// one, and a lane keeps the column sums of its experts in registers over the
// rows that it takes.  Counts are integer atomics in LDS, whose order changes
// nothing.  The gradient needs every row's counts, so there are three steps:
// sums of each workgroup's rows, their sum (in fp64 and in order) with the loss,
// and the gradient, which reads the logits again, from a cache in most sizes,
// and takes each row's softmax anew (kept, it would cost as many bytes).  Where
// one workgroup holds all rows at once the three are one kernel.
#include <algorithm>

#include "elements.hpp"
#include "router.hpp"
#include "rowloss_join.hpp"

namespace red {
namespace {

constexpr int kThreads = 1024; // a workgroup of the sums and of the gradient
constexpr double kLog2e64 = 1.4426950408889634074;
constexpr float kLn2f = 0.6931471805599453f;

struct RouterArgs {
    RouterCall c;
    float* prob_part;    // groups x E
    unsigned* count_part; // groups x E
    double* z_part;      // groups
    float* q;            // E
    uint32_t groups;
};

// Every lane of a row's GT neighbours gets their sum or maximum.  Up to 16 by
// DPP within a row of 16 lanes: neighbours, pairs, quads, eights.
template <class Op, int CTRL>
__device__ __forceinline__ float exchange(float v)
{
    const int u = __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true);
    return Op::apply(v, __int_as_float(u));
}
template <class Op, int GT>
__device__ __forceinline__ float group_reduce(float v)
{
    if constexpr (GT == kWave)
        return wave_reduce<Op>(v);
    v = exchange<Op, 0xb1>(v); // quad_perm 1 0 3 2
    v = exchange<Op, 0x4e>(v); // quad_perm 2 3 0 1
    if constexpr (GT == 16) {
        v = exchange<Op, 0x141>(v); // row_half_mirror
        v = exchange<Op, 0x140>(v); // row_mirror
    }
    return v;
}

template <class T, int GT, int NV>
struct RouterRow {
    static constexpr int W = T::W;
    uint32_t t, nvec, rest;
    __device__ __forceinline__ RouterRow(uint32_t E) : t(threadIdx.x % GT), nvec(E / W), rest(E % W) {}
    // Elements of the row, -inf past its end.
    __device__ __forceinline__ void load(const typename T::S* p, float (&f)[NV][W]) const
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = k * GT + t;
#pragma unroll
            for (int i = 0; i < W; ++i)
                f[k][i] = -INFINITY;
            if (j < nvec) {
                const u32x4u_t u = reinterpret_cast<const u32x4u_t*>(p)[j];
                T::unpack(u32x4_t{u.x, u.y, u.z, u.w}, f[k]);
            } else if (j == nvec) {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (i < (int)rest)
                        f[k][i] = T::widen(p[(size_t)nvec * W + i]);
            }
        }
    }
    __device__ __forceinline__ void store(typename T::S* p, const float (&f)[NV][W]) const
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = k * GT + t;
            if (j < nvec) {
                const u32x4_t v = T::pack(f[k]);
                reinterpret_cast<u32x4u_t*>(p)[j] = u32x4u_t{v.x, v.y, v.z, v.w};
            } else if (j == nvec) {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (i < (int)rest)
                        p[(size_t)nvec * W + i] = T::narrow(f[k][i]);
            }
        }
    }
};

// f becomes the exponentials 2^((z - max) log2 e); the row's sum and maximum.
// A row of -inf alone, or with a NaN or +inf, comes out as NaN.
template <int GT, int NV, int W>
__device__ __forceinline__ void exponentials(float (&f)[NV][W], float& max, float& sum)
{
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i)
            m = fmaxf(m, f[k][i]);
    max = m = group_reduce<OpMax, GT>(m);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) {
            f[k][i] = __builtin_amdgcn_exp2f((f[k][i] - m) * (float)kLog2e64);
            s += f[k][i];
        }
    sum = group_reduce<OpSum, GT>(s);
}

__device__ __forceinline__ float row_weight(const RouterCall& c, size_t r)
{
    return c.weight ? c.weight[r] : 1.0f / (float)c.m.rows;
}

// Step one, by every workgroup: its rows' sums to the workspace.
template <class T, int GT, int NV>
__device__ __forceinline__ void sum_rows(const RouterArgs& a, unsigned* lds_count, float* lds_prob)
{
    constexpr int W = T::W, RB = kThreads / GT;
    const RouterCall& c = a.c;
    const uint32_t E = (uint32_t)c.m.V;
    const RouterRow<T, GT, NV> at(E);
    __shared__ double lds_z[kThreads / kWave];
    for (uint32_t e = threadIdx.x; e < E; e += kThreads) {
        lds_count[e] = 0;
        lds_prob[e] = 0.0f;
    }
    __syncthreads();
    float acc[NV][W] = {};
    double zsum = 0.0;
    for (size_t r = (size_t)blockIdx.x * RB + threadIdx.x / GT; r < c.m.rows;
         r += (size_t)a.groups * RB) {
        const float w = row_weight(c, r);
        if (w == 0.0f)
            continue;
        float f[NV][W], m, s;
        at.load(static_cast<const typename T::S*>(c.m.z) + r * c.m.ld, f);
        for (uint32_t k = at.t; k < c.K; k += GT) {
            const int64_t e = c.experts[r * c.ldk + k];
            if (e >= 0 && e < (int64_t)E)
                atomicAdd(&lds_count[e], 1u);
        }
        exponentials<GT>(f, m, s);
        const float scale = w / s;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i)
                acc[k][i] += f[k][i] * scale;
        if (c.z != 0.0f && at.t == 0) {
            const double lse = m + __builtin_amdgcn_logf(s) * kLn2f;
            zsum += (double)w * lse * lse;
        }
    }
    // The lanes of a wave that own the same experts, then the waves in order.
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int d = GT; d < kWave; d *= 2)
                acc[k][i] += __shfl_xor(acc[k][i], d);
    zsum = wave_sum64(zsum);
    const uint32_t wave = threadIdx.x / kWave;
    if (threadIdx.x % kWave == 0)
        lds_z[wave] = zsum;
    for (uint32_t turn = 0; turn < kThreads / kWave; ++turn) {
        if (wave == turn && threadIdx.x % kWave < GT) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const uint32_t e = (k * GT + at.t) * W + i;
                    if (e < E)
                        lds_prob[e] += acc[k][i];
                }
        }
        __syncthreads();
    }
    for (uint32_t e = threadIdx.x; e < E; e += kThreads) {
        a.prob_part[(size_t)blockIdx.x * E + e] = lds_prob[e];
        a.count_part[(size_t)blockIdx.x * E + e] = lds_count[e];
    }
    if (threadIdx.x == 0) {
        double v = 0.0;
        for (int k = 0; k < kThreads / kWave; ++k)
            v += lds_z[k];
        a.z_part[blockIdx.x] = v;
    }
}

// Step two, by one workgroup: counts, probabilities, the loss and q.  Each
// expert's groups are added by several threads ("ways"), in order.
__device__ __forceinline__ void join_rows(const RouterArgs& a)
{
    const RouterCall& c = a.c;
    const uint32_t E = (uint32_t)c.m.V;
    __shared__ double lds_p[kThreads];
    __shared__ unsigned long long lds_n[kThreads];
    __shared__ unsigned long long lds_total[kThreads / kWave];
    __shared__ double lds_loss[kThreads / kWave];
    uint32_t cols = 4;
    while (cols < E && cols < kThreads)
        cols *= 2;
    const uint32_t ways = kThreads / cols, col = threadIdx.x % cols, way = threadIdx.x / cols;
    constexpr int kMost = (int)(kRouterExpertsMax / kThreads);
    double p[kMost];
    unsigned long long n[kMost], mine = 0;
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        p[k] = 0.0;
        n[k] = 0;
        const uint32_t e = k * kThreads + col;
        if (k * kThreads >= E)
            break;
        if (e < E) {
#pragma unroll 8
            for (uint32_t g = way; g < a.groups; g += ways) {
                p[k] += (double)a.prob_part[(size_t)g * E + e];
                n[k] += a.count_part[(size_t)g * E + e];
            }
        }
        __syncthreads();
        lds_p[threadIdx.x] = p[k];
        lds_n[threadIdx.x] = n[k];
        __syncthreads();
        if (way == 0 && e < E) {
            for (uint32_t v = 1; v < ways; ++v) {
                p[k] += lds_p[v * cols + col];
                n[k] += lds_n[v * cols + col];
            }
            c.counts[e] = (int64_t)n[k];
            if (c.prob)
                c.prob[e] = (float)p[k];
            mine += n[k];
        }
    }
    // The number of choices (integers), then the loss.
    for (int d = 1; d < kWave; d *= 2)
        mine += __shfl_xor(mine, d);
    if (threadIdx.x % kWave == 0)
        lds_total[threadIdx.x / kWave] = mine;
    __syncthreads();
    unsigned long long total = 0;
    for (int k = 0; k < kThreads / kWave; ++k)
        total += lds_total[k];
    const double b = (double)c.balance * (double)E;
    double part = 0.0;
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        const uint32_t e = k * kThreads + col;
        if (way == 0 && e < E) {
            const double q = total ? b * ((double)n[k] / (double)total) : 0.0;
            // Without a choice the probabilities have no part in the loss.
            part += total ? q * p[k] : 0.0;
            a.q[e] = (float)q;
        }
    }
    for (uint32_t g = threadIdx.x; g < a.groups; g += kThreads)
        if (c.z != 0.0f)
            part += (double)c.z * a.z_part[g];
    part = wave_sum64(part);
    if (threadIdx.x % kWave == 0)
        lds_loss[threadIdx.x / kWave] = part;
    __syncthreads();
    if (threadIdx.x == 0) {
        double loss = c.accum ? (double)c.loss[0] : 0.0;
        for (int k = 0; k < kThreads / kWave; ++k)
            loss += lds_loss[k];
        c.loss[0] = (float)loss;
    }
}

// Step three, by every workgroup: the gradient of its rows.
template <class T, int GT, int NV>
__device__ __forceinline__ void grad_rows(const RouterArgs& a, uint32_t groups)
{
    constexpr int W = T::W, RB = kThreads / GT;
    const RouterCall& c = a.c;
    const RouterRow<T, GT, NV> at((uint32_t)c.m.V);
    float q[NV][W];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t e = (k * GT + at.t) * W + i;
            q[k][i] = e < c.m.V ? a.q[e] : 0.0f;
        }
    for (size_t r = (size_t)blockIdx.x * RB + threadIdx.x / GT; r < c.m.rows;
         r += (size_t)groups * RB) {
        const float w = row_weight(c, r);
        float f[NV][W] = {};
        if (w != 0.0f) {
            float m, s, dot = 0.0f;
            at.load(static_cast<const typename T::S*>(c.m.z) + r * c.m.ld, f);
            exponentials<GT>(f, m, s);
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    dot += f[k][i] * q[k][i];
            dot = group_reduce<OpSum, GT>(dot);
            const float inverse = 1.0f / s;
            const float lse = m + __builtin_amdgcn_logf(s) * kLn2f;
            const float offset = 2.0f * c.z * lse - dot * inverse, scale = w * inverse;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    f[k][i] *= scale * (q[k][i] + offset);
        }
        at.store(static_cast<typename T::S*>(c.m.dz) + r * c.m.ldd, f);
    }
}

template <class T, int GT, int NV>
__global__ __launch_bounds__(kThreads) void router_sum_kernel(RouterArgs a)
{
    extern __shared__ unsigned lds[];
    sum_rows<T, GT, NV>(a, lds, reinterpret_cast<float*>(lds + a.c.m.V));
}

__global__ __launch_bounds__(kThreads) void router_join_kernel(RouterArgs a) { join_rows(a); }

template <class T, int GT, int NV>
__global__ __launch_bounds__(kThreads) void router_grad_kernel(RouterArgs a, uint32_t groups)
{
    grad_rows<T, GT, NV>(a, groups);
}

// All three by one workgroup, whose stores are seen by its own threads after a
// barrier.
template <class T, int GT, int NV>
__global__ __launch_bounds__(kThreads) void router_one_kernel(RouterArgs a)
{
    extern __shared__ unsigned lds[];
    sum_rows<T, GT, NV>(a, lds, reinterpret_cast<float*>(lds + a.c.m.V));
    __syncthreads();
    join_rows(a);
    __syncthreads();
    if (a.c.m.dz)
        grad_rows<T, GT, NV>(a, 1);
}

template <class T, int GT, int NV>
hipError_t launch(const RouterCall& c, const DeviceInfo& dev, const Workspace& ws, hipStream_t s)
{
    constexpr size_t RB = kThreads / GT;
    const size_t E = c.m.V, wanted = (c.m.rows + RB - 1) / RB;
    RouterArgs a = {c, nullptr, nullptr, nullptr, nullptr, 0};
    a.groups = (uint32_t)std::min(wanted, (size_t)std::min(dev.cus, 1024));
    char* p = static_cast<char*>(ws.partials);
    a.z_part = reinterpret_cast<double*>(p);
    p += sizeof(double) * 1024;
    a.q = reinterpret_cast<float*>(p);
    p += sizeof(float) * kRouterExpertsMax;
    a.groups = (uint32_t)std::min<size_t>(
        a.groups, (ws.partial_bytes - (p - static_cast<char*>(ws.partials))) / (8 * E));
    a.prob_part = reinterpret_cast<float*>(p);
    a.count_part = reinterpret_cast<unsigned*>(a.prob_part + (size_t)a.groups * E);
    const size_t lds = E * 8;
    if (a.groups == 1) {
        hipLaunchKernelGGL((router_one_kernel<T, GT, NV>), dim3(1), dim3(kThreads), lds, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((router_sum_kernel<T, GT, NV>), dim3(a.groups), dim3(kThreads), lds, s, a);
    hipLaunchKernelGGL(router_join_kernel, dim3(1), dim3(kThreads), 0, s, a);
    if (c.m.dz) {
        const uint32_t groups = (uint32_t)std::min(wanted, (size_t)dev.cus * 4);
        hipLaunchKernelGGL((router_grad_kernel<T, GT, NV>), dim3(groups), dim3(kThreads), 0, s, a,
                           groups);
    }
    return hipGetLastError();
}

// Lanes of a row and vectors of a lane, by the row's vectors.
template <class T>
hipError_t by_experts(const RouterCall& c, const DeviceInfo& dev, const Workspace& ws,
                      hipStream_t s)
{
    const size_t vecs = (c.m.V + T::W - 1) / T::W;
    if (vecs <= 4)
        return launch<T, 4, 1>(c, dev, ws, s);
    if (vecs <= 16)
        return launch<T, 16, 1>(c, dev, ws, s);
    if (vecs <= 32)
        return launch<T, 16, 2>(c, dev, ws, s);
    if (vecs <= 64)
        return launch<T, 64, 1>(c, dev, ws, s);
    if (vecs <= 128)
        return launch<T, 64, 2>(c, dev, ws, s);
    if (vecs <= 256)
        return launch<T, 64, 4>(c, dev, ws, s);
    if constexpr (T::W == 4)
        return launch<T, 64, 8>(c, dev, ws, s);
    return hipErrorInvalidValue; // not reached: E <= kRouterExpertsMax
}
static_assert(kRouterExpertsMax == 64 * 4 * 8, "the longest row's vectors");

} // namespace

hipError_t launch_router_balance(LogitType t, const RouterCall& a, const DeviceInfo& dev,
                                 const Workspace& ws, hipStream_t stream)
{
    switch (t) {
    case LogitType::F32: return by_experts<ElemF32>(a, dev, ws, stream);
    case LogitType::F16: return by_experts<ElemF16>(a, dev, ws, stream);
    default: return by_experts<ElemBF16>(a, dev, ws, stream);
    }
}

} // namespace red
