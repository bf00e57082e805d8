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
// The weight's gradient is a sum over rows: each thread keeps its columns' sums in
// fp32 registers over 64 of its rows at most, and adds those to fp64 sums of its own in
// LDS where it has more; a second kernel adds the workgroups' sums in fp64, in order.
// So a column's error does not grow with the rows.  No atomics: the result does not
// depend on timing.
//
// Bf16: 8192 x 8192 with a residual and 8 bits out 71.4 us a call, 6.6 TB/s; 1 x 4096 4.1,
// of which the host takes 3.3; the gradient of 16384 x 4096 95.1, 89 of them at 6.0 TB/s.
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

// A row's threads: 16 or 64 of a wave, or (GT 0) the whole workgroup, whose size
// the launch chooses.  Each holds NV vectors: vector k of thread t is number
// k threads + t.  Loads past the row's end go to a vector of zeros, without a
// branch, so that all are in flight at once; the elements after the last whole
// vector (`rest`) belong to the thread whose turn it is.
//
// STREAM: the rows are aligned to 16 bytes and pass the caches by.  (8192 x 8192
// bf16 with a residual and 8 bits out 72.5 us so, 81.1 otherwise, 80 with either
// loads or stores alone; unaligned rows, whose lines two loads share, were slower:
// 1531 x 5003 f32 20.8 against 16.9.)
template <class T, int GT, int NV, bool STREAM>
struct Row {
    static constexpr int W = T::W;
    uint32_t threads, t, nvec, rest;
    __device__ __forceinline__ Row(uint32_t D)
        : threads(GT ? GT : blockDim.x), t(GT ? threadIdx.x % GT : threadIdx.x), nvec(D / W),
          rest(D % W)
    {
    }

    __device__ __forceinline__ void load(const void* row, u32x4_t (&v)[NV]) const
    {
        load_as<STREAM>(row, v);
    }
    // What other workgroups read too.
    __device__ __forceinline__ void load_again(const void* row, u32x4_t (&v)[NV]) const
    {
        load_as<false>(row, v);
    }
    template <bool PASS>
    __device__ __forceinline__ void load_as(const void* row, u32x4_t (&v)[NV]) const
    {
        const typename T::S* p = static_cast<const typename T::S*>(row);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = k * threads + t;
            const u32x4u_t* at = j < nvec ? reinterpret_cast<const u32x4u_t*>(p) + j
                                          : reinterpret_cast<const u32x4u_t*>(&kZeroVec);
            u32x4u_t u;
            if constexpr (PASS)
                u = __builtin_nontemporal_load(at);
            else
                u = *at;
            v[k] = u32x4_t{u.x, u.y, u.z, u.w};
        }
        if (rest) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (k * threads + t == nvec)
                    v[k] = load_rest<T>(p + (size_t)nvec * W, rest, nvec > 0);
        }
    }
    // Vector k of the row.
    __device__ __forceinline__ void store(void* row, int k, const float (&f)[W]) const
    {
        typename T::S* p = static_cast<typename T::S*>(row);
        const uint32_t j = k * threads + t;
        const u32x4_t v = T::pack(f);
        if (j < nvec) {
            u32x4u_t* to = reinterpret_cast<u32x4u_t*>(p) + j;
            if constexpr (STREAM)
                __builtin_nontemporal_store(u32x4u_t{v.x, v.y, v.z, v.w}, to);
            else
                *to = u32x4u_t{v.x, v.y, v.z, v.w};
        } else if (rest && j == nvec) {
            store_rest<T>(p + (size_t)nvec * W, v, rest);
        }
    }
    __device__ __forceinline__ void store(void* row, const float (&f)[NV][W]) const
    {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            store(row, k, f[k]);
    }
    __device__ __forceinline__ void store8(uint8_t* p, const float (&f)[NV][W]) const
    {
        typedef unsigned word_t __attribute__((aligned(1)));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = k * threads + t;
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

// Sums and maxima over the threads of a row, in every one of them.  `lds` holds a
// value per wave; a use is followed by a barrier before the next.
constexpr int kMostWaves = 16;
template <int GT>
__device__ __forceinline__ double row_sum(double v, double* lds)
{
    if constexpr (GT && GT < kWave) {
#pragma unroll
        for (int d = GT / 2; d > 0; d /= 2)
            v += __shfl_xor(v, d);
        return v;
    } else {
        v = wave_sum64(v);
        if constexpr (GT == 0) {
            if (threadIdx.x % kWave == 0)
                lds[threadIdx.x / kWave] = v;
            __syncthreads();
            v = 0.0;
            for (uint32_t k = 0; k < blockDim.x / kWave; ++k)
                v += lds[k];
        }
        return v;
    }
}

template <int GT>
__device__ __forceinline__ float row_max(float v, float* lds)
{
    if constexpr (GT && GT < kWave) {
#pragma unroll
        for (int d = GT / 2; d > 0; d /= 2)
            v = fmaxf(v, __shfl_xor(v, d));
        return v;
    } else {
        v = wave_reduce<OpMax>(v);
        if constexpr (GT == 0) {
            if (threadIdx.x % kWave == 0)
                lds[threadIdx.x / kWave] = v;
            __syncthreads();
            v = lds[0];
            for (uint32_t k = 1; k < blockDim.x / kWave; ++k)
                v = fmaxf(v, lds[k]);
        }
        return v;
    }
}

// Whether a matrix's rows are all aligned to 16 bytes (ld: bytes).
struct Aligned {
    size_t rows;
    bool operator()(const void* p, size_t ld) const
    {
        return !p || ((uintptr_t)p % 16 == 0 && (rows == 1 || ld % 16 == 0));
    }
};

__device__ __forceinline__ float reciprocal_root(double ms) { return (float)(1.0 / sqrt(ms)); }

template <int GT>
constexpr int rows_per_block() { return GT ? kBlock / GT : 1; }
template <int GT>
constexpr int most_threads() { return GT ? kBlock : 1024; }

template <class T, int GT, int NV, bool STREAM>
__global__ __launch_bounds__(NV == 4 && T::W == 8 ? 512 : most_threads<GT>()) void
add_rmsnorm_kernel(NormCall a)
{
    constexpr int W = T::W, RB = rows_per_block<GT>();
    typedef typename T::S S;
    __shared__ double lds_sum[kMostWaves];
    __shared__ float lds_max[kMostWaves];
    const Row<T, GT, NV, STREAM> at((uint32_t)a.D);
    const size_t step = (size_t)gridDim.x * RB;
    for (size_t r = (size_t)blockIdx.x * RB + (GT ? threadIdx.x / (GT ? GT : 1) : 0); r < a.rows;
         r += step) {
        u32x4_t v[NV], w[NV];
        float f[NV][W];
        at.load(static_cast<const S*>(a.x) + r * a.ldx, v);
        if (a.residual) {
            u32x4_t u[NV];
            at.load(static_cast<const S*>(a.residual) + r * a.ldr, u);
            at.load_again(a.weight, w);
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
            at.load_again(a.weight, w);
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
        if constexpr (GT == 0)
            __syncthreads(); // before lds_sum and lds_max are written again
    }
}

// Rows whose terms a thread adds up in fp32.  (16384 x 4096 bf16 has 32 a thread,
// 262144 x 4096 512: 1590 us with an fp64 sum behind each 64 of them, 1594 without.)
constexpr uint32_t kRun = 64;
// fp64 sums of a thread in LDS and one more, so that neighbours' lie in other banks.
__host__ __device__ constexpr uint32_t fold_stride(uint32_t sums) { return sums + 1; }

struct GradArgs {
    NormGradCall c;
    float* partial; // a row of D column sums per workgroup; null: no weight gradient
    int last;       // one workgroup: it writes the gradient itself
    int folds;      // some thread has more than kRun rows
};

template <class T, int GT, int NV, bool STREAM>
__global__ __launch_bounds__((most_threads<GT>())) void rmsnorm_grad_kernel(GradArgs args)
{
    constexpr int W = T::W, RB = rows_per_block<GT>();
    typedef typename T::S S;
    const NormGradCall& a = args.c;
    __shared__ double lds_sum[2][kMostWaves];
    // A thread's column sums: in fp64 over its rows (folds), or in fp32 behind them
    // where rows share the workgroup.
    extern __shared__ double lds_fold[];
    const auto fold = [&](int k, int i) -> double& {
        return lds_fold[threadIdx.x * fold_stride(NV * W) + k * W + i];
    };
    const Row<T, GT, NV, STREAM> at((uint32_t)a.D);
    const size_t step = (size_t)gridDim.x * RB;
    // Four vectors a thread leave no registers for the weight between rows, nor for
    // the third input while a row's sum is waited for.
    constexpr bool kFull = NV == 4;
    u32x4_t w[NV];
    if (!kFull)
        at.load_again(a.weight, w);
    float acc[NV][W] = {};
    if (args.folds)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i)
                fold(k, i) = 0.0;
    uint32_t run = 0;
    int turn = 0;
    for (size_t r = (size_t)blockIdx.x * RB + (GT ? threadIdx.x / (GT ? GT : 1) : 0); r < a.rows;
         r += step) {
        u32x4_t hv[NV], gv[NV], sv[NV];
        at.load(static_cast<const S*>(a.h) + r * a.ldh, hv);
        at.load(static_cast<const S*>(a.dy) + r * a.lddy, gv);
        if (kFull)
            at.load_again(a.weight, w);
        if (!kFull && a.dsum)
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
        if (kFull && a.dsum)
            at.load(static_cast<const S*>(a.dsum) + r * a.ldds, sv);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float n[W], g[W], e[W], d[W];
            T::unpack(hv[k], n);
            T::unpack(gv[k], g);
            T::unpack(w[k], e);
#pragma unroll
            for (int i = 0; i < W; ++i)
                d[i] = (g[i] * e[i] - n[i] * rstd * mean) * rstd;
            if (a.dsum) {
                T::unpack(sv[k], e);
#pragma unroll
                for (int i = 0; i < W; ++i)
                    d[i] += e[i];
            }
            at.store(static_cast<S*>(a.dx) + r * a.lddx, k, d);
        }
        if (args.folds && ++run == kRun) {
            run = 0;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    fold(k, i) += (double)acc[k][i];
                    acc[k][i] = 0.0f;
                }
        }
    }
    if (!args.partial)
        return;
    float* out = args.last ? a.dweight : args.partial + (size_t)blockIdx.x * a.D;
    const auto put = [&](int k, int i, double sum) {
        const uint32_t j = (k * at.threads + at.t) * W + i;
        if (j < a.D)
            out[j] = (float)((args.last && a.accum ? (double)out[j] : 0.0) + sum);
    };
    // Rows that share a workgroup: their sums meet in its first row's threads.
    const uint32_t g = GT ? threadIdx.x / (GT ? GT : 1) : 0;
    if (args.folds) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i)
                fold(k, i) += (double)acc[k][i];
        if constexpr (RB > 1) {
            __syncthreads();
            if (g > 0)
                return;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                double sum = fold(k, i);
#pragma unroll
                for (int b = 1; b < RB; ++b)
                    sum += lds_fold[(b * GT + at.t) * fold_stride(NV * W) + k * W + i];
                put(k, i, sum);
            }
        return;
    }
    if constexpr (RB > 1) {
        float* lds_acc = reinterpret_cast<float*>(lds_fold);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i)
                lds_acc[(k * W + i) * kBlock + threadIdx.x] = acc[k][i];
        __syncthreads();
        if (g > 0)
            return;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int b = 1; b < RB; ++b)
                    acc[k][i] += lds_acc[(k * W + i) * kBlock + b * GT + at.t];
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i)
            put(k, i, (double)acc[k][i]);
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

// Waves of the gradient kernel for each compute unit: about what fits at once, and
// no more, since each workgroup leaves a row of column sums.  (16384 x 4096 bf16:
// 95.7 us with 16, 108 with 32.  Fewer, with the next row requested ahead, took 97.8
// and needed twice the registers.)
constexpr unsigned kGradWavesPerCu = 16;

template <class T, int GT, int NV>
struct Shape {
    // Threads of a workgroup for rows of `vecs` vectors.
    static unsigned threads(size_t vecs)
    {
        return GT ? (unsigned)kBlock : (unsigned)(((vecs + NV - 1) / NV + kWave - 1) / kWave * kWave);
    }
    static hipError_t norm(const NormCall& a, size_t vecs, hipStream_t s)
    {
        constexpr size_t RB = rows_per_block<GT>();
        const unsigned groups = (unsigned)std::min((a.rows + RB - 1) / RB, size_t(1) << 20);
        const Aligned al = {a.rows};
        if (al(a.x, a.ldx * sizeof(typename T::S)) && al(a.residual, a.ldr * sizeof(typename T::S)) &&
            al(a.sum, a.lds * sizeof(typename T::S)) && al(a.y, a.ldy * sizeof(typename T::S)))
            hipLaunchKernelGGL((add_rmsnorm_kernel<T, GT, NV, true>), dim3(groups),
                               dim3(threads(vecs)), 0, s, a);
        else
            hipLaunchKernelGGL((add_rmsnorm_kernel<T, GT, NV, false>), dim3(groups),
                               dim3(threads(vecs)), 0, s, a);
        return hipGetLastError();
    }
    static hipError_t grad(const NormGradCall& a, size_t vecs, const DeviceInfo& dev,
                           const Workspace& ws, hipStream_t s)
    {
        constexpr size_t RB = rows_per_block<GT>();
        size_t groups = (a.rows + RB - 1) / RB;
        groups = std::min(groups, (size_t)dev.cus *
                                      std::max(1u, kGradWavesPerCu * kWave / threads(vecs)));
        if (a.dweight)
            groups = std::min(groups, ws.partial_bytes / (a.D * sizeof(float)));
        GradArgs args = {a, a.dweight ? static_cast<float*>(ws.partials) : nullptr, 0, 0};
        if (a.dweight && groups == 1) {
            args.last = 1;
            args.partial = a.dweight;
        }
        args.folds = a.dweight && (a.rows + groups * RB - 1) / (groups * RB) > kRun;
        // At most 136 KiB for the waves that a compute unit gets.
        const size_t of = threads(vecs);
        const unsigned lds = (unsigned)(args.folds ? of * fold_stride(NV * T::W) * sizeof(double)
                                        : a.dweight && RB > 1 ? of * NV * T::W * sizeof(float)
                                                              : 0);
        const Aligned al = {a.rows};
        if (al(a.h, a.ldh * sizeof(typename T::S)) && al(a.dy, a.lddy * sizeof(typename T::S)) &&
            al(a.dsum, a.ldds * sizeof(typename T::S)) && al(a.dx, a.lddx * sizeof(typename T::S)))
            hipLaunchKernelGGL((rmsnorm_grad_kernel<T, GT, NV, true>), dim3((unsigned)groups),
                               dim3(threads(vecs)), lds, s, args);
        else
            hipLaunchKernelGGL((rmsnorm_grad_kernel<T, GT, NV, false>), dim3((unsigned)groups),
                               dim3(threads(vecs)), lds, s, args);
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

// The threads that share a row and the vectors of each.  The gradient, and the norm
// of few rows, whose time is that of one row, take one vector a thread as far as
// that goes ("wide"); the norm of many two, or four where a row is long (8192 x 8192
// bf16: 1024 threads with one 134 us, 512 with two 75.7, 256 with four 72.5).
template <class T, class F>
hipError_t by_wide_shape(size_t vecs, F f)
{
    if (vecs <= 16)
        return f(Shape<T, 16, 1>(), vecs);
    if (vecs <= 64)
        return f(Shape<T, 64, 1>(), vecs);
    if (vecs <= 1024)
        return f(Shape<T, 0, 1>(), vecs);
    if constexpr (T::W == 4)
        if (vecs > 2048)
            return f(Shape<T, 0, 4>(), vecs);
    return f(Shape<T, 0, 2>(), vecs);
}
template <class T, class F>
hipError_t by_shape(bool wide, size_t D, F f)
{
    const size_t vecs = (D + T::W - 1) / T::W;
    if (wide || vecs <= 64)
        return by_wide_shape<T>(vecs, f);
    if (vecs <= 128)
        return f(Shape<T, 64, 2>(), vecs);
    if (vecs <= 640)
        return f(Shape<T, 0, 2>(), vecs);
    return f(Shape<T, 0, 4>(), vecs);
}
template <class T, class F>
hipError_t by_grad_shape(size_t D, F f)
{
    const size_t vecs = (D + T::W - 1) / T::W;
    // A wave a row needs no barrier (12572 x 259 f32: 23.3 us, 31.5 with two waves).
    if (vecs > 64 && vecs <= 128)
        return f(Shape<T, 64, 2>(), vecs);
    return by_wide_shape<T>(vecs, f);
}
static_assert(kNormColsMax == 1024 * 4 * 4 && kNormColsMax == 1024 * 2 * 8 &&
                  kNormColsMax == 512 * 4 * 8,
              "the longest row's vectors");

} // namespace

hipError_t launch_add_rmsnorm(LogitType t, const NormCall& a, const DeviceInfo& dev,
                              hipStream_t stream)
{
    const bool wide = a.rows <= (size_t)dev.cus;
    const auto f = [&](auto shape, size_t vecs) { return shape.norm(a, vecs, stream); };
    switch (t) {
    case LogitType::F32: return by_shape<ElemF32>(wide, a.D, f);
    case LogitType::F16: return by_shape<ElemF16>(wide, a.D, f);
    default: return by_shape<ElemBF16>(wide, a.D, f);
    }
}

hipError_t launch_rmsnorm_grad(LogitType t, const NormGradCall& a, const DeviceInfo& dev,
                               const Workspace& ws, hipStream_t stream)
{
    const auto f = [&](auto shape, size_t vecs) { return shape.grad(a, vecs, dev, ws, stream); };
    switch (t) {
    case LogitType::F32: return by_grad_shape<ElemF32>(a.D, f);
    case LogitType::F16: return by_grad_shape<ElemF16>(a.D, f);
    default: return by_grad_shape<ElemBF16>(a.D, f);
    }
}

} // namespace red
