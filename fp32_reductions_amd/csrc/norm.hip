// norm.hip -- the root-mean-square norm of rows and its gradient.
//
//     h = x + residual,  rstd = (mean h^2 + eps)^(-1/2),  y = h rstd w
//     n = h rstd,  g = dy w:  dx = (g - n mean(g n)) rstd + dsum,
//                             dw = sum over rows of dy n
//
// A row stays in the registers of the threads that share it between its
// statistics and its outputs, so each input is read once and each output
// written once: HBM bounds it where rows are many, one row's chain of
// latencies where they are few.  Rows are widened to fp32; the sums over a row
// are fp64 (a square of 1e30 or 1e-30 has its place there, and two fp64 steps
// an element hide behind the loads); every output is rounded once, and y is
// computed from the sum before its rounding.
//
// The weight's gradient is a sum over rows: each workgroup keeps its columns'
// sums in fp32 registers over the rows that it takes, a fixed few dozen where
// rows are many, and a second kernel adds the workgroups' sums in fp64, in
// order.  No atomics: the result does not depend on timing.
#include <algorithm>

#include "elements.hpp"
#include "norm.hpp"
#include "rowloss_join.hpp"

namespace red {
namespace {

// 8-bit floats of 4 exponent bits (no infinities, largest 448).
constexpr float kE4m3Max = 448.0f;
// Below this the reciprocal of a row's scale would not be finite: such a row is
// a row of zeros in 8 bits.
constexpr float kTiny8 = 1.0e-35f;

__device__ const u32x4_t kZeroVec = {0, 0, 0, 0};

// Row elements of GT threads with NV vectors each: vector k of thread t is
// number k GT + t.  Loads past the row's end go to a vector of zeros, without a
// branch, so that all are in flight at once.
template <class T, int GT, int NV>
struct Row {
    static constexpr int W = T::W;
    uint32_t t, nvec, rest; // rest: elements after the whole vectors
    __device__ __forceinline__ Row(uint32_t D) : t(threadIdx.x % GT), nvec(D / W), rest(D % W) {}

    __device__ __forceinline__ void load(const void* row, u32x4_t (&v)[NV]) const
    {
        const typename T::S* p = static_cast<const typename T::S*>(row);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = k * GT + t;
            const u32x4u_t* at = j < nvec ? reinterpret_cast<const u32x4u_t*>(p) + j
                                          : reinterpret_cast<const u32x4u_t*>(&kZeroVec);
            const u32x4u_t u = *at;
            v[k] = u32x4_t{u.x, u.y, u.z, u.w};
        }
        if (rest) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (k * GT + t == nvec) {
                    float f[W];
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        f[i] = i < (int)rest ? T::widen(p[(size_t)nvec * W + i]) : 0.0f;
                    v[k] = T::pack(f);
                }
        }
    }
    __device__ __forceinline__ void store(void* row, const float (&f)[NV][W]) const
    {
        typename T::S* p = static_cast<typename T::S*>(row);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = k * GT + t;
            if (j < nvec) {
                const u32x4_t v = T::pack(f[k]);
                *(reinterpret_cast<u32x4u_t*>(p) + j) = u32x4u_t{v.x, v.y, v.z, v.w};
            } else if (rest && j == nvec) {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (i < (int)rest)
                        p[(size_t)nvec * W + i] = T::narrow(f[k][i]);
            }
        }
    }
    __device__ __forceinline__ void store8(uint8_t* p, const float (&f)[NV][W]) const
    {
        typedef unsigned word_t __attribute__((aligned(1)));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = k * GT + t;
            unsigned q[W / 4];
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                int b = __builtin_amdgcn_cvt_pk_fp8_f32(f[k][4 * i], f[k][4 * i + 1], 0, false);
                q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(f[k][4 * i + 2], f[k][4 * i + 3], b, true);
            }
            if (j < nvec) {
#pragma unroll
                for (int i = 0; i < W / 4; ++i)
                    reinterpret_cast<word_t*>(p + (size_t)j * W)[i] = q[i];
            } else if (rest && j == nvec) {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (i < (int)rest)
                        p[(size_t)nvec * W + i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
            }
        }
    }
};

// Sums and maxima over the GT threads of a row, in every one of them.  `lds`
// holds a value per wave; a use is followed by a barrier before the next.
template <int GT>
__device__ __forceinline__ double row_sum(double v, double* lds)
{
    if constexpr (GT < kWave) {
#pragma unroll
        for (int d = GT / 2; d > 0; d /= 2)
            v += __shfl_xor(v, d);
        return v;
    } else {
        v = wave_sum64(v);
        if constexpr (GT > kWave) {
            if (threadIdx.x % kWave == 0)
                lds[threadIdx.x / kWave] = v;
            __syncthreads();
            v = 0.0;
#pragma unroll
            for (int k = 0; k < GT / kWave; ++k)
                v += lds[k];
        }
        return v;
    }
}

template <int GT>
__device__ __forceinline__ float row_max(float v, float* lds)
{
    if constexpr (GT < kWave) {
#pragma unroll
        for (int d = GT / 2; d > 0; d /= 2)
            v = fmaxf(v, __shfl_xor(v, d));
        return v;
    } else {
        v = wave_reduce<OpMax>(v);
        if constexpr (GT > kWave) {
            if (threadIdx.x % kWave == 0)
                lds[threadIdx.x / kWave] = v;
            __syncthreads();
            v = lds[0];
#pragma unroll
            for (int k = 1; k < GT / kWave; ++k)
                v = fmaxf(v, lds[k]);
        }
        return v;
    }
}

__device__ __forceinline__ float reciprocal_root(double ms) { return (float)(1.0 / sqrt(ms)); }

template <int GT>
constexpr int rows_per_block() { return GT < kBlock ? kBlock / GT : 1; }

template <class T, int GT, int NV>
__global__ __launch_bounds__(GT < kBlock ? kBlock : GT) void add_rmsnorm_kernel(NormCall a)
{
    constexpr int W = T::W, RB = rows_per_block<GT>(), WAVES = GT > kWave ? GT / kWave : 1;
    typedef typename T::S S;
    __shared__ double lds_sum[WAVES];
    __shared__ float lds_max[WAVES];
    const Row<T, GT, NV> at((uint32_t)a.D);
    const size_t step = (size_t)gridDim.x * RB;
    for (size_t r = (size_t)blockIdx.x * RB + threadIdx.x / GT; r < a.rows; r += step) {
        u32x4_t v[NV], w[NV];
        float f[NV][W];
        at.load(static_cast<const S*>(a.x) + r * a.ldx, v);
        if (a.residual) {
            u32x4_t u[NV];
            at.load(static_cast<const S*>(a.residual) + r * a.ldr, u);
            at.load(a.weight, w);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float e[W];
                T::unpack(v[k], f[k]);
                T::unpack(u[k], e);
#pragma unroll
                for (int i = 0; i < W; ++i)
                    f[k][i] += e[i];
            }
        } else {
            at.load(a.weight, w);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                T::unpack(v[k], f[k]);
        }
        double ss = 0.0;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i)
                ss = __builtin_fma((double)f[k][i], (double)f[k][i], ss);
        ss = row_sum<GT>(ss, lds_sum);
        const float rstd = reciprocal_root(ss / (double)a.D + (double)a.eps);
        // The row's inputs are in registers: outputs may lie over them.
        if (a.sum)
            at.store(static_cast<S*>(a.sum) + r * a.lds, f);
        if (a.rstd && at.t == 0)
            a.rstd[r] = rstd;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float e[W];
            T::unpack(w[k], e);
#pragma unroll
            for (int i = 0; i < W; ++i)
                f[k][i] = f[k][i] * rstd * e[i];
        }
        if (a.y)
            at.store(static_cast<S*>(a.y) + r * a.ldy, f);
        if (a.y8) {
            float most = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    most = fmaxf(most, fabsf(f[k][i]));
            most = row_max<GT>(most, lds_max);
            if (most < kTiny8)
                most = 0.0f;
            const float inverse = most > 0.0f ? kE4m3Max / most : 0.0f;
            if (at.t == 0)
                a.scale8[r] = most / kE4m3Max;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    f[k][i] *= inverse;
            at.store8(a.y8 + r * a.ldy8, f);
        }
        if constexpr (GT > kWave)
            __syncthreads(); // before lds_sum and lds_max are written again
    }
}

struct GradArgs {
    NormGradCall c;
    float* partial; // a row of D column sums per workgroup; null: no weight gradient
    int last;       // one workgroup: it writes the gradient itself
};

template <class T, int GT, int NV>
__global__ __launch_bounds__(GT < kBlock ? kBlock : GT) void rmsnorm_grad_kernel(GradArgs args)
{
    constexpr int W = T::W, RB = rows_per_block<GT>(), WAVES = GT > kWave ? GT / kWave : 1;
    typedef typename T::S S;
    const NormGradCall& a = args.c;
    __shared__ double lds_sum[2][WAVES];
    const Row<T, GT, NV> at((uint32_t)a.D);
    const size_t step = (size_t)gridDim.x * RB;
    u32x4_t w[NV];
    at.load(a.weight, w);
    float acc[NV][W] = {};
    int turn = 0;
    for (size_t r = (size_t)blockIdx.x * RB + threadIdx.x / GT; r < a.rows; r += step) {
        u32x4_t hv[NV], gv[NV], sv[NV];
        at.load(static_cast<const S*>(a.h) + r * a.ldh, hv);
        at.load(static_cast<const S*>(a.dy) + r * a.lddy, gv);
        if (a.dsum)
            at.load(static_cast<const S*>(a.dsum) + r * a.ldds, sv);
        const float rstd = a.rstd[r];
        double c = 0.0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float n[W], g[W], e[W];
            T::unpack(hv[k], n);
            T::unpack(gv[k], g);
            T::unpack(w[k], e);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                n[i] *= rstd;
                acc[k][i] += g[i] * n[i];
                c = __builtin_fma((double)(g[i] * e[i]), (double)n[i], c);
            }
        }
        c = row_sum<GT>(c, lds_sum[turn]);
        turn ^= 1; // the next row's sums go elsewhere: no second barrier
        const float mean = (float)(c / (double)a.D);
        float d[NV][W];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float n[W], g[W], e[W];
            T::unpack(hv[k], n);
            T::unpack(gv[k], g);
            T::unpack(w[k], e);
#pragma unroll
            for (int i = 0; i < W; ++i)
                d[k][i] = (g[i] * e[i] - n[i] * rstd * mean) * rstd;
            if (a.dsum) {
                T::unpack(sv[k], e);
#pragma unroll
                for (int i = 0; i < W; ++i)
                    d[k][i] += e[i];
            }
        }
        at.store(static_cast<S*>(a.dx) + r * a.lddx, d);
    }
    if (!args.partial)
        return;
    // Rows that share a workgroup: their sums meet in its first row's threads.
    if constexpr (RB > 1) {
        __shared__ float lds_acc[RB][GT * NV * W];
        const uint32_t g = threadIdx.x / GT;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i)
                lds_acc[g][(k * W + i) * GT + at.t] = acc[k][i];
        __syncthreads();
        if (g > 0)
            return;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int b = 1; b < RB; ++b)
                    acc[k][i] += lds_acc[b][(k * W + i) * GT + at.t];
    }
    float* out = args.last ? a.dweight : args.partial + (size_t)blockIdx.x * a.D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const uint32_t first = (k * GT + at.t) * W;
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (first + i < a.D)
                out[first + i] =
                    (args.last && a.accum ? out[first + i] : 0.0f) + acc[k][i];
    }
}

// dweight[j] = [dweight[j] +] the sum of n partial rows: 64 columns a
// workgroup, 16 threads a column, each adding every sixteenth row in order.
constexpr int kSumCols = 64, kSumWays = 16;
__global__ __launch_bounds__(kSumCols* kSumWays) void
column_finish_kernel(const float* __restrict__ partial, uint32_t n, uint32_t D, float* dweight,
                     int accum)
{
    __shared__ double lds[kSumWays][kSumCols];
    const uint32_t col = threadIdx.x % kSumCols, way = threadIdx.x / kSumCols;
    const uint32_t j = blockIdx.x * kSumCols + col;
    double v = 0.0;
    if (j < D) {
#pragma unroll 8
        for (uint32_t b = way; b < n; b += kSumWays)
            v += (double)partial[(size_t)b * D + j];
    }
    lds[way][col] = v;
    __syncthreads();
    if (way || j >= D)
        return;
#pragma unroll
    for (int k = 1; k < kSumWays; ++k)
        v += lds[k][col];
    dweight[j] = (float)((accum ? (double)dweight[j] : 0.0) + v);
}

// Workgroups of the gradient kernel: enough to fill the device twice over, and
// no more, since each leaves a row of column sums.
constexpr unsigned kGradGroupsPerCu = 2;

template <class T, int GT, int NV>
struct Shape {
    static constexpr int kThreads = GT < kBlock ? kBlock : GT;
    static hipError_t norm(const NormCall& a, const DeviceInfo&, hipStream_t s)
    {
        constexpr size_t RB = rows_per_block<GT>();
        const size_t groups = std::min((a.rows + RB - 1) / RB, size_t(1) << 20);
        hipLaunchKernelGGL((add_rmsnorm_kernel<T, GT, NV>), dim3((unsigned)groups),
                           dim3(kThreads), 0, s, a);
        return hipGetLastError();
    }
    static hipError_t grad(const NormGradCall& a, const DeviceInfo& dev, const Workspace& ws,
                           hipStream_t s)
    {
        constexpr size_t RB = rows_per_block<GT>();
        size_t groups = (a.rows + RB - 1) / RB;
        groups = std::min(groups, (size_t)dev.cus * kGradGroupsPerCu * (1024 / kThreads));
        if (a.dweight)
            groups = std::min(groups, ws.partial_bytes / (a.D * sizeof(float)));
        GradArgs args = {a, a.dweight ? static_cast<float*>(ws.partials) : nullptr, 0};
        if (a.dweight && groups == 1) {
            args.last = 1;
            args.partial = a.dweight;
        }
        hipLaunchKernelGGL((rmsnorm_grad_kernel<T, GT, NV>), dim3((unsigned)groups),
                           dim3(kThreads), 0, s, args);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || !a.dweight || groups == 1)
            return e;
        hipLaunchKernelGGL(column_finish_kernel,
                           dim3((unsigned)((a.D + kSumCols - 1) / kSumCols)),
                           dim3(kSumCols * kSumWays), 0, s, static_cast<const float*>(ws.partials),
                           (uint32_t)groups, (uint32_t)a.D, a.dweight, a.accum);
        return hipGetLastError();
    }
};

// The threads that share a row: up to four vectors each.  Few rows get one
// vector a thread, as far as that goes: what counts then is one row's time.
template <class T, class F>
hipError_t by_shape(size_t rows, size_t D, const DeviceInfo& dev, F f)
{
    const size_t vecs = (D + T::W - 1) / T::W;
    const bool few = rows <= (size_t)dev.cus;
    if (vecs <= 16)
        return f(Shape<T, 16, 1>());
    if (vecs <= 64)
        return f(Shape<T, 64, 1>());
    if (vecs <= 128 && !few)
        return f(Shape<T, 64, 2>());
    if (vecs <= 256)
        return f(Shape<T, 256, 1>());
    if (few && vecs <= 1024)
        return f(Shape<T, 1024, 1>());
    if (vecs <= 512)
        return f(Shape<T, 256, 2>());
    if (vecs <= 1024)
        return f(Shape<T, 256, 4>());
    if (few && vecs <= 2048)
        return f(Shape<T, 1024, 2>());
    if (vecs <= 2048)
        return f(Shape<T, 512, 4>());
    if constexpr (T::W == 4)
        return f(Shape<T, 1024, 4>());
    return hipErrorInvalidValue; // not reached: D <= kNormColsMax
}
static_assert(kNormColsMax == 4096 * 4 && kNormColsMax == 2048 * 8, "the longest row's vectors");

} // namespace

#define RED_NORM_BY_TYPE(t, call)                       \
    switch (t) {                                        \
    case LogitType::F32: return by_shape<ElemF32> call; \
    case LogitType::F16: return by_shape<ElemF16> call; \
    default: return by_shape<ElemBF16> call;            \
    }

hipError_t launch_add_rmsnorm(LogitType t, const NormCall& a, const DeviceInfo& dev,
                              hipStream_t stream)
{
    const auto f = [&](auto shape) { return shape.norm(a, dev, stream); };
    RED_NORM_BY_TYPE(t, (a.rows, a.D, dev, f))
}

hipError_t launch_rmsnorm_grad(LogitType t, const NormGradCall& a, const DeviceInfo& dev,
                               const Workspace& ws, hipStream_t stream)
{
    const auto f = [&](auto shape) { return shape.grad(a, dev, ws, stream); };
    RED_NORM_BY_TYPE(t, (a.rows, a.D, dev, f))
}

} // namespace red
