// rowloss_kernels.hpp -- losses over rows of logits: kernels and launches,
// instantiated once per element type.
//
// Every operator here reduces a row z[0..V) of logits to
//
//     m = max z,   S = sum 2^((z - m) c),   U = sum 2^((z - m) c) (z - m) c,
//
// with c = scale * log2(e), so that p_v = 2^((z_v - m) c) / S is the softmax
// of the scaled row, ln S + scale * m its log-sum-exp and ln S - ln 2 * U / S
// its entropy.  The gradient of each row loss with respect to the logits is
//
//     dz_v = 2^((z_v - m) c) (A + B (z_v - m) c) + (terms in a few columns)
//
// with A and B from the loss of that row alone.  So a loss and its gradient
// need one read of the row and one write: row_kernel keeps the row in the
// registers of its workgroup between the two.  What bounds it is HBM where
// rows are many (at 16 bits the vector unit is busy in half of the cycles with a
// gradient, where an element is unpacked three times and has two exponentials,
// and in nine of ten where an entropy alone is wanted), and the chain of one
// row's latencies where they are few.
//
// Statistics are fp32 per thread (sums of at most a few hundred terms, then
// a tree); what is computed once per row (logarithms, ratios, losses) is
// fp64, so that a sum of thousands of log-probabilities keeps its last bits.
// Terms below 2^-126 of a row's largest count as zero (v_exp_f32); where a
// result rests on some columns alone (distillation's rest) they are summed
// against their own largest.
//
// Determinism: no atomics on results; every sum has a fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "rowloss.hpp"
#include "rowloss_pairs.hpp"

namespace red {

// ---- element types ---------------------------------------------------------
//
// Vec holds W elements in 16 bytes.  pack rounds each value once, to nearest
// even.
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

struct ElemF32 {
    typedef float S;
    static constexpr int W = 4;
    static constexpr unsigned kNegInf = 0xff800000u;
    static __device__ __forceinline__ void unpack(const u32x4_t& v, float (&f)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = __uint_as_float(v[i]);
    }
    static __device__ __forceinline__ u32x4_t pack(const float (&f)[4])
    {
        u32x4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __float_as_uint(f[i]);
        return v;
    }
    static __device__ __forceinline__ float widen(S s) { return s; }
    static __device__ __forceinline__ S narrow(float f) { return f; }
};

struct ElemF16 {
    typedef uint16_t S;
    static constexpr int W = 8;
    static constexpr unsigned kNegInf = 0xfc00fc00u;
    static __device__ __forceinline__ void unpack(const u32x4_t& v, float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f16x2_t h = __builtin_bit_cast(f16x2_t, (unsigned)v[i]);
            f[2 * i] = (float)h.x;
            f[2 * i + 1] = (float)h.y;
        }
    }
    static __device__ __forceinline__ u32x4_t pack(const float (&f)[8])
    {
        u32x4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f16x2_t h;
            h.x = (_Float16)f[2 * i];
            h.y = (_Float16)f[2 * i + 1];
            v[i] = __builtin_bit_cast(unsigned, h);
        }
        return v;
    }
    static __device__ __forceinline__ float widen(S s)
    {
        return (float)__builtin_bit_cast(_Float16, s);
    }
    static __device__ __forceinline__ S narrow(float f)
    {
        return __builtin_bit_cast(S, (_Float16)f);
    }
};

struct ElemBF16 {
    typedef uint16_t S;
    static constexpr int W = 8;
    static constexpr unsigned kNegInf = 0xff80ff80u;
    static __device__ __forceinline__ void unpack(const u32x4_t& v, float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float((unsigned)v[i] << 16);
            f[2 * i + 1] = __uint_as_float((unsigned)v[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ u32x4_t pack(const float (&f)[8])
    {
        u32x4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x2_t p;
            p.x = f[2 * i];
            p.y = f[2 * i + 1];
            v[i] = __builtin_bit_cast(unsigned, __builtin_convertvector(p, bf16x2_t));
        }
        return v;
    }
    static __device__ __forceinline__ float widen(S s)
    {
        return __uint_as_float((unsigned)s << 16);
    }
    static __device__ __forceinline__ S narrow(float f)
    {
        return __builtin_bit_cast(S, (__bf16)f);
    }
};

namespace rowloss {

constexpr double kLog2e = 1.4426950408889634074;
constexpr double kLn2 = 0.69314718055994530942;
// Exponents are clamped here where they multiply a probability, so that a
// probability of zero (a logit of -inf) contributes 0 and not 0 * inf.
constexpr float kLowest = -1.0e30f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// ---- a row's elements and the threads that own them ------------------------
//
// `head` elements up to the first 16-byte boundary, `nvec` vectors, and the
// rest.  Vector j belongs to thread j mod GT of the row's GT threads; the
// head and the rest (at most 2 (W - 1) <= 14 elements) go one each to the
// first threads.
struct Span {
    uint32_t head, nvec, tail, singles;
    template <class T>
    static __device__ __forceinline__ Span of(const typename T::S* row, uint32_t V)
    {
        Span s;
        const uint32_t past = (uint32_t)((uintptr_t)row & 15u) / (uint32_t)sizeof(typename T::S);
        const uint32_t head = past ? T::W - past : 0;
        s.head = head < V ? head : V;
        s.nvec = (V - s.head) / T::W;
        s.tail = s.head + s.nvec * T::W;
        s.singles = s.head + (V - s.tail);
        return s;
    }
    __device__ __forceinline__ uint32_t single(uint32_t t) const
    {
        return t < head ? t : t - head + tail;
    }
};

// A gradient row need not share its logits' alignment: gfx950 stores
// unaligned 16-byte vectors to global memory.
typedef unsigned u32x4u_t __attribute__((ext_vector_type(4), aligned(2)));

typedef __attribute__((address_space(1))) const u32x4_t global_vec;

template <bool STREAM>
__device__ __forceinline__ u32x4_t load_vec(global_vec* p)
{
    if constexpr (STREAM)
        return __builtin_nontemporal_load(p);
    else
        return *p;
}

__device__ __forceinline__ void store_vec(void* p, const u32x4_t& v)
{
    u32x4u_t u;
    u.x = v.x; u.y = v.y; u.z = v.z; u.w = v.w;
    __builtin_nontemporal_store(u, reinterpret_cast<u32x4u_t*>(p));
}

// Loads past a row's end go to a vector of -inf, which adds nothing to any
// statistic, instead of being skipped.
template <class T>
__device__ const u32x4_t kNegInfVec = {T::kNegInf, T::kNegInf, T::kNegInf, T::kNegInf};

// The vectors j = first + k GT + t (k < NV) of a row, in this order and
// without a branch between them, so that the first can be used while the last
// is on its way (with a branch around each load the compiler waits for all).
template <class T, int GT, int NV, bool STREAM>
__device__ __forceinline__ void load_chunk(const u32x4_t* base, uint32_t first, uint32_t nvec,
                                           uint32_t t, u32x4_t (&v)[NV])
{
    global_vec* none = (global_vec*)&kNegInfVec<T>;
    asm volatile("" : "+v"(t)); // no offset is kept from here to the stores
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const uint32_t j = first + k * GT + t;
        v[k] = load_vec<STREAM>(j < nvec ? (global_vec*)base + j : none);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// ---- statistics ------------------------------------------------------------
struct Stat {
    float m, s, u;
};

// The reference of an exponent: the maximum, or 0 while every element so far
// is -inf (whose terms then come out as 0).
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }

// The exponent of an element is one fused step, z c - shift, with shift the
// rounded product of the reference and c.  What that rounding drops (delta =
// ref c - shift, exact in one fused step) is a factor 2^-delta common to all
// of a thread's terms, put back once per chunk.  Where shift is so large that
// delta is no small number any more (a row filled with its type's lowest
// value, say), the difference z - ref is taken first.
constexpr float kWideShift = 1048576.0f; // delta below 2^-4
__device__ __forceinline__ bool is_wide(float shift) { return !(fabsf(shift) < kWideShift); }

// What the statistics leave out: nothing, or the columns of a bitmap with one
// bit per element and W bits per vector.  They are left out of the maximum
// too: a listed logit 90 above all others would take every other term below
// 2^-126 of itself, and the columns outside would have no sum of their own.
struct TakeAll {
    static constexpr bool kSome = false;
    __device__ __forceinline__ unsigned skip(uint32_t) const { return 0; }
    __device__ __forceinline__ bool skip_one(uint32_t) const { return false; }
};

template <int W>
struct TakeUnmarked {
    static constexpr bool kSome = true;
    const uint32_t* bits;
    uint32_t nvec, singles; // singles: a bit for each element outside the vectors
    __device__ __forceinline__ unsigned skip(uint32_t j) const
    {
        const uint32_t at = (j < nvec ? j : 0) * W; // past the row's end nothing is lost
        return (reinterpret_cast<const unsigned char*>(bits)[at >> 3] >> (at & 7)) & ((1u << W) - 1);
    }
    __device__ __forceinline__ bool skip_one(uint32_t t) const { return (singles >> t) & 1; }
};

// Elements with a bit in `skip` become -inf, which adds nothing to any
// statistic.
template <class T>
__device__ __forceinline__ void drop(u32x4_t& v, unsigned skip)
{
    constexpr int kPerWord = T::W / 4;
#pragma unroll
    for (int i = 0; i < T::W; ++i) {
        const unsigned lanes = kPerWord == 1 ? 0xffffffffu : 0xffffu << (i % kPerWord * 16);
        const unsigned mask = (skip >> i) & 1 ? lanes : 0u;
        v[i / kPerWord] = (v[i / kPerWord] & ~mask) | (T::kNegInf & mask);
    }
}

// Folds the NG vectors first + k GT + t and the single element `one` (-inf:
// none) into st: first the maximum, then the sums against it.
template <class T, int GT, int NG, bool ENT>
__device__ __forceinline__ void fold_group(const u32x4_t (&v)[NG], uint32_t first, uint32_t nvec,
                                           float one, bool skip_one, float c, Stat& st)
{
    constexpr int W = T::W;
    float m0 = fmaxf(st.m, one), m1 = -INFINITY;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        if (k && first + k * GT >= nvec)
            break;
        float f[W];
        T::unpack(v[k], f);
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            m0 = fmaxf(fmaxf(m0, f[i]), f[i + 1]);
            m1 = fmaxf(fmaxf(m1, f[i + 2]), f[i + 3]);
        }
    }
    const float m = fmaxf(m0, m1);
    const float ref = reference(m), mc = ref * c;
    // What was summed against the old maximum moves to the new one.
    const float d = fmaxf((st.m - ref) * c, kLowest), r = exp2_fast(d);
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[2] = {0.0f, 0.0f};
    const bool wide = is_wide(mc);
    auto sums = [&](auto exponent) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            if (k && first + k * GT >= nvec)
                break;
            float f[W];
            T::unpack(v[k], f);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float x = exponent(f[i]), e = exp2_fast(x);
                s[i & 3] += e;
                if constexpr (ENT)
                    u[i & 1] = fmaf(e, fmaxf(x, kLowest), u[i & 1]);
            }
        }
        if (!skip_one) {
            const float x = exponent(one), e = exp2_fast(x);
            s[1] += e;
            if constexpr (ENT)
                u[1] = fmaf(e, fmaxf(x, kLowest), u[1]);
        }
    };
    if (__builtin_expect(wide, 0))
        sums([&](float z) { return (z - ref) * c; });
    else
        sums([&](float z) { return fmaf(z, c, -mc); });
    const float delta = wide ? 0.0f : fmaf(ref, c, -mc), back = exp2_fast(-delta);
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    if constexpr (ENT)
        st.u = fmaf(r, fmaf(st.s, d, st.u), back * fmaf(-delta, sum, u[0] + u[1]));
    st.s = fmaf(st.s, r, back * sum);
    st.m = m;
}

// Folds a chunk of NV vectors and one single element, kFold vectors at a
// time: while the first are folded the others are still on their way.  What
// `take` leaves out is -inf in v afterwards: the gradient of those columns is
// written from elsewhere.
constexpr int kFold = 8;
template <class T, int GT, int NV, bool ENT, class Take>
__device__ __forceinline__ void fold_chunk(u32x4_t (&v)[NV], uint32_t first, uint32_t nvec,
                                           uint32_t t, float one, bool skip_one, float c,
                                           const Take& take, Stat& st)
{
    constexpr int NG = NV < kFold ? NV : kFold;
    static_assert(NV % NG == 0, "whole groups");
#pragma unroll
    for (int g = 0; g < NV; g += NG) {
        if (g && first + g * GT >= nvec)
            break;
        if constexpr (Take::kSome) {
            unsigned skips[NG];
#pragma unroll
            for (int k = 0; k < NG; ++k)
                skips[k] = take.skip(first + (g + k) * GT + t);
#pragma unroll
            for (int k = 0; k < NG; ++k)
                if (__builtin_amdgcn_ballot_w64(skips[k] != 0)) {
                    asm volatile(""); // a branch that few waves take, not selects for all
                    drop<T>(v[g + k], skips[k]);
                }
        }
        u32x4_t part[NG];
#pragma unroll
        for (int k = 0; k < NG; ++k)
            part[k] = v[g + k];
        fold_group<T, GT, NG, ENT>(part, first + g * GT, nvec, g || skip_one ? -INFINITY : one,
                                   g ? true : skip_one, c, st);
    }
}

// Moves st to the maximum m (>= st.m).
template <bool ENT>
__device__ __forceinline__ void move_to(Stat& st, float m, float c)
{
    const float d = fmaxf((st.m - reference(m)) * c, kLowest), r = exp2_fast(d);
    if constexpr (ENT)
        st.u = r * fmaf(st.s, d, st.u);
    st.s *= r;
    st.m = m;
}

// The statistics of a row from those of its GT threads, in every thread.
// lds: 3 floats per wave of a group of more than one.
template <int GT, bool ENT>
__device__ __forceinline__ Stat combine(Stat st, float c, float* lds)
{
    move_to<ENT>(st, wave_reduce<OpMax>(st.m), c);
    st.s = wave_reduce<OpSum>(st.s);
    if constexpr (ENT)
        st.u = wave_reduce<OpSum>(st.u);
    if constexpr (GT > kWave) {
        constexpr int kParts = GT / kWave;
        const int w = (threadIdx.x % GT) / kWave;
        if ((threadIdx.x & 63) == 0) {
            lds[w] = st.m;
            lds[kParts + w] = st.s;
            if constexpr (ENT)
                lds[2 * kParts + w] = st.u;
        }
        __syncthreads();
        const uint32_t lane = threadIdx.x & 63;
        st = {-INFINITY, 0.0f, 0.0f};
        if (lane < kParts) {
            st.m = lds[lane];
            st.s = lds[kParts + lane];
            if constexpr (ENT)
                st.u = lds[2 * kParts + lane];
        }
        move_to<ENT>(st, wave_reduce<OpMax>(st.m), c);
        st.s = wave_reduce<OpSum>(st.s);
        if constexpr (ENT)
            st.u = wave_reduce<OpSum>(st.u);
    }
    return st;
}

// dz = 2^x (A + B x) for every element of a row.
struct Slope {
    float a, b;
};

template <bool ENT>
__device__ __forceinline__ float slope_at(float x, const Slope& k)
{
    const float e = exp2_fast(x);
    if constexpr (ENT)
        return e * fmaf(k.b, fmaxf(x, kLowest), k.a);
    else
        return e * k.a;
}

// The exponent x of a logit against the row's maximum; `lost` is what the
// fused form's shift leaves out of it (delta above).
struct Exponent {
    float ref, c, shift, lost;
    bool wide;
    __device__ __forceinline__ Exponent(float reference_, float c_) : ref(reference_), c(c_)
    {
        shift = ref * c;
        wide = is_wide(shift);
        lost = wide ? 0.0f : fmaf(ref, c, -shift);
    }
    __device__ __forceinline__ float at(float z) const { return (z - ref) * c; }
    // A + B x in terms of the exponent that leaves `lost` out.
    __device__ __forceinline__ Slope fused(const Slope& k) const
    {
        const float back = exp2_fast(-lost);
        return {back * fmaf(-lost, k.b, k.a), back * k.b};
    }
};

template <class T, int GT, int NV, bool ENT>
__device__ __forceinline__ void write_chunk(const u32x4_t (&v)[NV], typename T::S* out,
                                            uint32_t first, uint32_t nvec, uint32_t t,
                                            const Exponent& ex, const Slope& exact_slope)
{
    constexpr int W = T::W;
    const Slope slope = ex.fused(exact_slope);
    auto put = [&](auto exponent) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k && first + k * GT >= nvec)
                break;
            const uint32_t j = first + k * GT + t;
            float f[W];
            T::unpack(v[k], f);
#pragma unroll
            for (int i = 0; i < W; ++i)
                f[i] = slope_at<ENT>(exponent(f[i]), slope);
            if (j < nvec)
                store_vec(out + (size_t)j * W, T::pack(f));
        }
    };
    if (__builtin_expect(ex.wide, 0))
        put([&](float z) { return (z - ex.ref) * ex.c; });
    else
        put([&](float z) { return fmaf(z, ex.c, -ex.shift); });
}

template <class T, int GT>
__device__ __forceinline__ void write_zeros(typename T::S* row, const Span& sp, uint32_t t)
{
    for (uint32_t j = t; j < sp.nvec; j += GT)
        store_vec(row + sp.head + (size_t)j * T::W, u32x4_t{0, 0, 0, 0});
    if (t < sp.singles)
        row[sp.single(t)] = 0;
}

// ---- the operators ---------------------------------------------------------
//
// An operator has: kEntropy (U is needed), kList (its row has a teacher's
// list), Args, Row (what it loads of a row before its logits: `live` says
// whether the row counts at all, `y` its target column), and
//   done(row, stat, zy, leader): outputs of the row (by the leader alone),
//     and the slope of its gradient;
//   fix: what is added to the gradient in the target's column.

// values[row], or `other` without values; a branch around the load would put
// one memory latency after another before the row's own loads, so then
// something else that has a value for each row is read.
__device__ __forceinline__ float value_or(const float* values, float other, const float* something,
                                          size_t row)
{
    const float v = (values ? values : something)[row];
    return values ? v : other;
}

// The fp64 part of a row: ln p of a logit, and the entropy.
struct RowLogs {
    double ln_s, scale, ref;
    __device__ __forceinline__ RowLogs(const Stat& st, float scale_)
        : ln_s(log((double)st.s)), scale(scale_), ref(reference(st.m))
    {
    }
    __device__ __forceinline__ double logp(float z) const { return ((double)z - ref) * scale - ln_s; }
    __device__ __forceinline__ double lse() const { return ref * scale + ln_s; }
    __device__ __forceinline__ double entropy(const Stat& st) const
    {
        return ln_s - kLn2 * ((double)st.u / (double)st.s);
    }
};

// What a row's gradient takes from its statistics, where another kernel
// writes it: dz_v = 2^((z_v - ref) c) (a + b (z_v - ref) c), and fix more in the
// target's column.  All zero for a row that does not count.
struct RowSlope {
    float ref, a, b, fix;
};

// Log-probability of the target, log-sum-exp and entropy.
template <bool ENT>
struct LogprobOp {
    static constexpr bool kEntropy = ENT, kList = false, kHasGrad = false;
    struct Args {
        const int64_t* targets;
        float *logp, *lse, *entropy;
        float scale;
    };
    struct Row {
        bool live, hit;
        uint32_t y;
    };
    static __device__ __forceinline__ Row begin(const Args& a, size_t row, uint32_t V)
    {
        const int64_t y = a.targets[row];
        const bool hit = (uint64_t)y < V;
        return {true, hit, hit ? (uint32_t)y : 0u};
    }
    static __device__ __forceinline__ Slope done(const Args& a, const Row& r, size_t row,
                                                 const Stat& st, float zy, bool leader, float& fix)
    {
        if (leader) {
            const RowLogs l(st, a.scale);
            a.logp[row] = r.hit ? (float)l.logp(zy) : 0.0f;
            a.lse[row] = (float)l.lse();
            if constexpr (ENT)
                a.entropy[row] = (float)l.entropy(st);
        }
        fix = 0.0f;
        return {0.0f, 0.0f};
    }
    static __device__ __forceinline__ void dead(const Args&, size_t, bool) {}
    static __device__ __forceinline__ NoJoin join(const Args&, const Row&) { return {}; }
};

// First pass of the preference loss: maximum, sum and log-probability.
// JOIN: the wave that comes last in a pair finishes the pair (PairJoin), which
// takes twice the registers.
template <bool JOIN>
struct PreferenceOp {
    static constexpr bool kEntropy = false, kList = false, kHasGrad = false;
    struct Args {
        float2* stat;
        PairArgs pair;
    };
    struct Row {
        bool live;
        uint32_t y;
        int64_t start; // this lane's bound of a sequence
    };
    static __device__ __forceinline__ Row begin(const Args& a, size_t row, uint32_t V)
    {
        const uint32_t lane = threadIdx.x & 63, last = 2 * a.pair.pairs;
        const int64_t y = a.pair.targets[row];
        const bool hit = (uint64_t)y < V;
        return {hit, hit ? (uint32_t)y : 0u,
                JOIN ? a.pair.starts[lane < last ? lane : last] : 0};
    }
    static __device__ __forceinline__ Slope done(const Args& a, const Row&, size_t row,
                                                 const Stat& st, float zy, bool leader, float& fix)
    {
        if (leader) {
            const RowLogs l(st, 1.0f);
            a.stat[row] = make_float2(st.m, st.s);
            put(a, row, l.logp(zy));
        }
        fix = 0.0f;
        return {0.0f, 0.0f};
    }
    static __device__ __forceinline__ void dead(const Args& a, size_t row, bool leader)
    {
        if (leader) {
            a.stat[row] = make_float2(0.0f, 1.0f);
            put(a, row, 0.0);
        }
    }
    // The slope of a row that no sequence has is 0.
    static __device__ __forceinline__ void put(const Args& a, size_t row, double logp)
    {
        store_shared(a.pair.row_logp + row, logp);
        if (!JOIN)
            a.pair.row_slope[row] = 0.0f;
    }
    static __device__ __forceinline__ auto join(const Args& a, const Row& r)
    {
        if constexpr (JOIN)
            return PairJoin(a.pair, r.start);
        else
            return NoJoin();
    }
};

// Clipped policy loss.  With r = exp(logp - old), d = ref - logp:
//   loss  = -min(r A, clip(r) A) + kl (exp(d) - d - 1) - ent H
//   slope = -(r A where r A <= clip(r) A, else 0) + kl (1 - exp(d))   (to logp)
// and d logp / dz_v = scale (delta_vy - p_v), dH / dz_v = -scale p_v (ln p_v + H).
template <bool ENT>
struct PolicyOp {
    static constexpr bool kEntropy = ENT, kList = false, kHasGrad = true;
    struct Args {
        const int64_t* targets;
        const float *old_logp, *ref_logp, *advantage, *weight;
        double clip_min, clip_max, kl, ent;
        float scale, mean;
        float *logp, *entropy;
        Join join;
    };
    struct Row {
        bool live;
        uint32_t y;
        float weight, old_logp, advantage, ref_logp;
    };
    static __device__ __forceinline__ Row begin(const Args& a, size_t row, uint32_t V)
    {
        const int64_t y = a.targets[row];
        const float w = value_or(a.weight, a.mean, a.old_logp, row);
        const bool hit = (uint64_t)y < V;
        return {hit && w != 0.0f, hit ? (uint32_t)y : 0u, w, a.old_logp[row], a.advantage[row],
                value_or(a.ref_logp, 0.0f, a.old_logp, row)};
    }
    static __device__ __forceinline__ Slope done(const Args& a, const Row& r, size_t row,
                                                 const Stat& st, float zy, bool leader, float& fix)
    {
        const RowLogs l(st, a.scale);
        const double logp = l.logp(zy), adv = r.advantage, w = r.weight;
        // Even lanes take the ratio's exponential, odd ones the KL term's.
        const double d = a.ref_logp ? (double)r.ref_logp - logp : 0.0;
        const double e = exp(threadIdx.x & 1 ? d : logp - (double)r.old_logp);
        const double ratio = __shfl(e, 0);
        const double free = ratio * adv;
        const double bound = ratio < a.clip_min   ? a.clip_min
                             : ratio > a.clip_max ? a.clip_max
                                                  : ratio;
        const double clipped = bound * adv;
        // Not (free > clipped), so that a NaN stays one.
        double loss = free > clipped ? -clipped : -free;
        double g = free > clipped ? 0.0 : -free;
        if (a.ref_logp) {
            // In fp64 the difference is off by 2^-53, below a loss's last bit.
            const double k = __shfl(e, 1) - 1.0;
            loss += a.kl * (k - d);
            g -= a.kl * k;
        }
        double H = 0.0;
        if constexpr (ENT) {
            H = l.entropy(st);
            loss -= a.ent * H;
        }
        if (leader) {
            a.logp[row] = (float)logp;
            if (ENT && a.entropy)
                a.entropy[row] = (float)H;
            a.join.put(row, w * loss);
        }
        const double gw = w * g * l.scale;
        fix = (float)gw;
        Slope k = {(float)(-gw / (double)st.s), 0.0f};
        if constexpr (ENT) {
            const double hw = w * a.ent * l.scale / (double)st.s;
            k.a = (float)(-gw / (double)st.s + hw * (H - l.ln_s));
            k.b = (float)(hw * kLn2);
        }
        return k;
    }
    static __device__ __forceinline__ void dead(const Args& a, size_t row, bool leader)
    {
        if (leader) {
            a.logp[row] = 0.0f;
            if (ENT && a.entropy)
                a.entropy[row] = 0.0f;
            a.join.put(row, 0.0);
        }
    }
    static __device__ __forceinline__ Join join(const Args& a, const Row&) { return a.join; }
};

// Divergence from a teacher's largest logits.  S: the columns listed, q_k
// the teacher's probability of entry k, Q their sum and, with TAIL, q_r =
// 1 - Q the rest's, against p_r = sum of p outside S:
//   loss = sum_k q_k (ln q_k - ln p_k) [+ q_r (ln q_r - ln p_r)]
//   dz_v = w scale (p_v (Q + q_r) - q_v) in S,
//          w scale p_v (Q + q_r - q_r / p_r) outside
// (Q and no second term without TAIL).
template <bool TAIL>
struct DistillOp {
    static constexpr bool kEntropy = false, kList = true, kTail = TAIL, kHasGrad = true;
    struct Args {
        const int64_t* idx;
        const float *val, *teacher_lse, *weight;
        uint32_t K;
        size_t ldk;
        float scale, mean;
        float* row_loss_out;
        Join join;
    };
    struct Row {
        bool live;
        float weight, teacher_lse;
    };
    static __device__ __forceinline__ Row begin(const Args& a, size_t row, uint32_t)
    {
        const float w = value_or(a.weight, a.mean, a.val, row);
        return {w != 0.0f, w, TAIL ? a.teacher_lse[row] : 0.0f};
    }
    static __device__ __forceinline__ void dead(const Args& a, size_t row, bool leader)
    {
        if (leader) {
            a.join.put(row, 0.0);
            if (a.row_loss_out)
                a.row_loss_out[row] = 0.0f;
        }
    }
    static __device__ __forceinline__ Join join(const Args& a, const Row&) { return a.join; }
};

// What rounding can leave of 1 - Q where the teacher has nothing outside its
// list: teacher_lse is an fp32 number (2^-24 of itself) from a sum of up to V
// exponentials, and comes in as sixteen such steps at most.  Where the student
// has nothing there either (masked columns: e^x is 0 even in fp64, for the
// largest of them against the row's largest), such a rest counts as 0, and not
// as infinitely far from the student.
constexpr double kRestRounding = 0x1p-20, kNoTerm = -745.2;
constexpr float kFar = 0x1p-100f;

// A row's teacher in LDS: its columns (-1: padding; the high bit marks the
// later ones of a column listed more than once), probabilities, the logits
// in those columns, and a bit for each listed column.
struct TeacherLds {
    uint32_t* bits;
    int* col;
    float* q;
    float* z;
    double* cross; // sum q (ln q - scale (z - ref)), ref the reference of the largest logit listed
    double* sum;   // Q
    int* state;    // [0]: the row has a teacher; [1]: the largest logit listed
    uint32_t* marked; // of each wave: the columns it marked; the high bit: one of them twice
    static constexpr size_t kHead = 32 + 16 * 4;
    static __host__ __device__ size_t bytes(size_t words, size_t K)
    {
        return (kHead + 4 * words + 12 * K + 15) / 16 * 16;
    }
    __device__ __forceinline__ TeacherLds(char* base, uint32_t words, uint32_t K)
    {
        cross = reinterpret_cast<double*>(base);
        sum = cross + 1;
        state = reinterpret_cast<int*>(base + 16);
        marked = reinterpret_cast<uint32_t*>(base + 32);
        bits = reinterpret_cast<uint32_t*>(base + kHead);
        col = reinterpret_cast<int*>(bits + words);
        q = reinterpret_cast<float*>(col + K);
        z = q + K;
    }
};

template <class Op>
__device__ __forceinline__ uint32_t list_length(const typename Op::Args& a)
{
    if constexpr (Op::kList)
        return a.K;
    else
        return 0;
}

// Words of the bitmap of V columns: a bit for each element of a vector, in the
// order of the vectors, and one word for the elements outside.
inline __host__ __device__ uint32_t bitmap_words(uint32_t V) { return (V + 31) / 32 + 1; }

// A value that is the same in all lanes of a wave, in scalar registers: a row's
// few fp64 numbers beside its vectors would cost a wave per SIMD.
__device__ __forceinline__ float uniform(float v)
{
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
}
__device__ __forceinline__ double uniform(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = __builtin_amdgcn_readfirstlane((int)(unsigned)b);
    const unsigned hi = __builtin_amdgcn_readfirstlane((int)(unsigned)(b >> 32));
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}

// LDS written by one lane of a wave and read by another of the same wave.
__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Reads the row's list.  Every wave marks the columns in its own vectors, in
// words of its own (64 vectors after one another are 64 W bits): so no wave
// waits for another before it folds.  The first wave also keeps the list:
// columns, their logits and the student's logits in them.  The columns are
// loaded before the row's vectors, which would otherwise return first, and
// used when the last of those is under way (4096 rows of 131072 bf16, 64
// entries and the rest: 412 us with one wave that marks for all, 384 so).
template <class T, int GT>
struct ListReader {
    typedef typename T::S S;
    static constexpr uint32_t kBatch = 2, kStep = kBatch * kWave;
    const TeacherLds& l;
    const Span& sp;
    const int64_t* idx;
    const float* val;
    const S* z;
    uint32_t V, K, words, wave, lane;
    uint32_t k0 = 0, listed = 0;
    bool again = false;
    bool taught = false; // first wave: this lane has an entry above -inf, or a NaN
    float top_val = -INFINITY, top_z = -INFINITY; // first wave: this lane's largest
    int64_t at[kBatch];
    float v[kBatch];
    S zk[kBatch];

    __device__ __forceinline__ void load()
    {
#pragma unroll
        for (uint32_t b = 0; b < kBatch; ++b) {
            const uint32_t k = k0 + b * kWave + lane;
            at[b] = idx[k < K ? k : 0];
            v[b] = val[k < K && wave == 0 ? k : 0]; // no branch: it would wait for the load
        }
        if (k0 == 0)
            clear();
#pragma unroll
        for (uint32_t b = 0; b < kBatch; ++b) {
            at[b] = k0 + b * kWave + lane < K && (uint64_t)at[b] < V ? at[b] : -1;
            zk[b] = z[at[b] < 0 || wave != 0 ? 0 : at[b]];
        }
    }
    // The wave's words of the bitmap.
    __device__ __forceinline__ void clear()
    {
        constexpr uint32_t kWords = kWave * T::W / 32; // of 64 vectors
        const uint32_t rounds = (sp.nvec + GT - 1) / GT;
        for (uint32_t i = lane; i < rounds * kWords; i += kWave) {
            const uint32_t word = (i / kWords * GT + wave * kWave) * T::W / 32 + i % kWords;
            if (word < words - 1)
                l.bits[word] = 0;
        }
        if (wave == 0 && lane == 0)
            l.bits[words - 1] = 0;
        wave_lds_fence();
    }
    __device__ __forceinline__ void use()
    {
#pragma unroll
        for (uint32_t b = 0; b < kBatch; ++b) {
            if (wave == 0) {
                const uint32_t k = k0 + b * kWave + lane;
                const float logit = at[b] < 0 ? -INFINITY : T::widen(zk[b]);
                const float value = at[b] < 0 ? -INFINITY : v[b];
                if (k < K) {
                    l.col[k] = (int)at[b];
                    l.q[k] = value;
                    l.z[k] = logit;
                }
                taught |= !(value == -INFINITY);
                top_val = fmaxf(top_val, value);
                top_z = fmaxf(top_z, logit);
            }
            if (at[b] < 0)
                continue;
            const uint32_t e = (uint32_t)at[b];
            uint32_t place, owner = 0;
            if (e >= sp.head && e < sp.tail) {
                place = e - sp.head;
                owner = place / T::W % GT / kWave;
            } else {
                place = (words - 1) * 32 + (e < sp.head ? e : e - sp.tail + sp.head);
            }
            if (owner == wave) {
                const uint32_t bit = 1u << (place & 31);
                const bool seen = atomicOr(&l.bits[place >> 5], bit) & bit;
                again |= seen;
                listed += !seen;
            }
        }
    }
    // All but the last entries, whose loads are left under way.
    __device__ __forceinline__ void begin()
    {
        for (load(); k0 + kStep < K; load()) {
            use();
            k0 += kStep;
        }
    }
    // The last, and what the wave has found.
    __device__ __forceinline__ void end()
    {
        use();
        uint32_t n = (uint32_t)wave_reduce<OpSum>((float)listed);
        n |= __any(again) ? 0x80000000u : 0u;
        if (lane == 0)
            l.marked[wave] = n;
        wave_lds_fence();
    }
};

// The same wave turns the list into the teacher's probabilities and the sums
// of the row's loss.  fp64: a row's loss is a small difference of these sums.
template <class T, bool TAIL>
__device__ __forceinline__ void weigh_teacher(const typename DistillOp<TAIL>::Args& a,
                                              const typename DistillOp<TAIL>::Row& r,
                                              bool taught, float top, float top_z,
                                              uint32_t lane, const TeacherLds& l)
{
    taught = __any(taught);
    top = wave_reduce<OpMax>(top);
    top_z = wave_reduce<OpMax>(top_z);
    const float ref = reference(top_z);
    wave_lds_fence();
    const double scale = a.scale;
    double shift, first_q = 0.0; // first_q: the probability of this lane's first entry
    if constexpr (TAIL) {
        shift = r.teacher_lse;
    } else {
        double s = 0.0;
        const double most = reference(top);
        for (uint32_t k = lane; k < a.K; k += kWave) {
            const double e = exp(((double)l.q[k] - most) * scale);
            first_q = k == lane ? e : first_q;
            s += e;
        }
        s = wave_sum64(s);
        shift = most * scale + log(s);
        first_q /= s;
    }
    double sum = 0.0, cross = 0.0;
    for (uint32_t k = lane; k < a.K; k += kWave) {
        const double lq = (double)l.q[k] * scale - shift;
        const double q = !TAIL && k == lane ? first_q : exp(lq);
        const int col = l.col[k];
        l.q[k] = col >= 0 ? (float)q : 0.0f;
        if (col < 0)
            continue;
        sum += q;
        if (q != 0.0) // an entry of no probability adds nothing, whatever its logit
            cross += q * (lq - ((double)l.z[k] - (double)ref) * scale);
    }
    sum = wave_sum64(sum);
    cross = wave_sum64(cross);
    if (lane == 0) {
        *l.sum = sum;
        *l.cross = cross;
        l.state[0] = TAIL || taught;
        l.state[1] = __float_as_int(top_z);
    }
    wave_lds_fence();
}

// Where a column is listed more than once its first entry takes the sum of the
// probabilities, and the others are marked.  One wave.
__device__ __forceinline__ void merge_entries(uint32_t K, uint32_t lane, const TeacherLds& l)
{
    for (uint32_t k = lane; k < K; k += kWave) {
        const int col = l.col[k] & 0x7fffffff;
        if (col == 0x7fffffff)
            continue;
        uint32_t first = k;
        float q = 0.0f;
        for (uint32_t j = 0; j < K; ++j)
            if ((l.col[j] & 0x7fffffff) == col) {
                first = j < first ? j : first;
                q += l.q[j];
            }
        if (first == k)
            l.q[k] = q;
        else
            l.col[k] = col | (int)0x80000000;
    }
    wave_lds_fence();
}

// ---- one read and one write per row ----------------------------------------
//
// GT threads share a row (64: four rows per workgroup of 256).  Thread t
// holds vectors t, t + GT, ... of the row, NV of them; MULTI rows are longer
// than that and come in chunks of GT NV vectors, of which the last one read
// is still there when the gradient is written and the others are read again
// (from the caches: the rows in flight on 256 compute units fit there).
// GRAD: the gradient is written.
//
// Measured (bf16, us a call): policy loss of 8192 rows of 131072, a quarter of
// them masked, 653 (5.7 TB/s; 639 without arithmetic), of 1024 rows of 32768
// 26, of 96 rows 8.7; log-probability and entropy of 4096 rows of 131072 166
// (6.5 TB/s).
template <class T, int GT, int NV, bool MULTI, bool GRAD, class Op>
__global__ __launch_bounds__(GT < 256 ? 256 : GT) void row_kernel(
    const typename T::S* z, typename T::S* dz, uint32_t rows, uint32_t V, size_t ld, size_t ldd,
    float c, typename Op::Args args)
{
    typedef typename T::S S;
    constexpr int kRowsPerGroup = GT < 256 ? 256 / GT : 1;
    extern __shared__ __align__(16) char dynamic_lds[];
    __shared__ float parts[GT > kWave ? 3 * (GT / kWave) : 1];
    const uint32_t t = threadIdx.x % GT;
    const uint32_t group = __builtin_amdgcn_readfirstlane(threadIdx.x / GT);
    const uint32_t row = blockIdx.x * kRowsPerGroup + group;
    if (row >= rows)
        return; // whole waves; a group of more than one wave has a row
    const S* zr = z + (size_t)row * ld;
    S* dr = GRAD ? dz + (size_t)row * ldd : nullptr;
    const bool leader = t == 0;
    const Span sp = Span::of<T>(zr, V);
    const typename Op::Row r = Op::begin(args, row, V);
    auto join = Op::join(args, r);
    auto dead_row = [&]() __attribute__((always_inline)) {
        Op::dead(args, row, leader);
        const unsigned before = t < kWave ? join.arrive(row) : 0;
        if constexpr (GRAD)
            write_zeros<T, GT>(dr, sp, t);
        if (t < kWave)
            join.finish(before, row, rows);
    };
    if (!r.live) {
        dead_row();
        return;
    }
    const u32x4_t* vec = reinterpret_cast<const u32x4_t*>(zr + sp.head);
    constexpr uint32_t kChunk = GT * NV;
    const uint32_t chunks = MULTI ? (sp.nvec + kChunk - 1) / kChunk : 1;
    const uint32_t words = Op::kList ? bitmap_words(V) : 0;
    const uint32_t K = list_length<Op>(args);
    const TeacherLds l(dynamic_lds + group * TeacherLds::bytes(words, K), words, K);
    ListReader<T, GT> list = {l, sp, nullptr, nullptr, zr, V, K, words, t / kWave, t % kWave};
    if constexpr (Op::kList) {
        list.idx = args.idx + row * args.ldk;
        list.val = args.val + row * args.ldk;
        list.begin();
    }
    // Loads return in the order of their issue: the single elements first, or
    // the fold of the first vectors would wait for the last.
    const bool has_one = t < sp.singles;
    const uint32_t at_one = has_one ? sp.single(t) : 0;
    const S raw_one = zr[at_one];
    S raw_zy = 0;
    if constexpr (!Op::kList)
        raw_zy = zr[r.y];
    u32x4_t v[NV];
    // Every load of the row (of its first chunk) is under way before the
    // first is used.
    load_chunk<T, GT, NV, !(MULTI && GRAD)>(vec, 0, sp.nvec, t, v);
    const float one = has_one ? T::widen(raw_one) : -INFINITY;

    Stat st = {-INFINITY, 0.0f, 0.0f};
    float zy = 0.0f;
    auto fold_row = [&](bool skip, const auto& take) __attribute__((always_inline)) {
        fold_chunk<T, GT, NV, Op::kEntropy>(v, 0, sp.nvec, t, one, skip, c, take, st);
        if constexpr (MULTI)
            for (uint32_t ch = 1; ch < chunks; ++ch) {
                load_chunk<T, GT, NV, !GRAD>(vec, ch * kChunk, sp.nvec, t, v);
                fold_chunk<T, GT, NV, Op::kEntropy>(v, ch * kChunk, sp.nvec, t, -INFINITY, true, c,
                                                    take, st);
            }
    };
    if constexpr (Op::kList) {
        list.end();
        if (t < kWave)
            weigh_teacher<T, Op::kTail>(args, r, list.taught, list.top_val, list.top_z, t, l);
        if constexpr (Op::kTail) {
            const TakeUnmarked<T::W> take{l.bits, sp.nvec, has_one ? l.bits[words - 1] : 0u};
            fold_row(has_one && take.skip_one(t), take);
        } else {
            fold_row(false, TakeAll{});
        }
    } else {
        zy = T::widen(raw_zy);
        fold_row(false, TakeAll{});
    }
    st = combine<GT, Op::kEntropy>(st, c, parts);
    const Exponent ex(reference(st.m), c);

    Slope slope;
    float fix = 0.0f, factor = 0.0f, mass = 0.0f;
    float listed_ref = 0.0f, listed_sum = 0.0f; // for the columns listed
    if constexpr (Op::kList) {
        const int taught = l.state[0];
        const float top_z = __int_as_float(l.state[1]);
        const double Q = uniform(*l.sum);
        if (!taught) { // no teacher: the row does not count
            dead_row();
            return;
        }
        uint32_t listed = 0, again = 0;
#pragma unroll
        for (int w = 0; w < GT / kWave; ++w) {
            listed += l.marked[w] & 0x7fffffffu;
            again |= l.marked[w] & 0x80000000u;
        }
        if (__builtin_amdgcn_readfirstlane(again)) {
            if (t < kWave)
                merge_entries(args.K, t, l);
            if constexpr (GT > kWave)
                __syncthreads();
        }
        // Of the whole row: the largest logit and the sum against it.  With the
        // rest, st holds the columns outside alone, against their own maximum.
        const float top = Op::kTail ? fmaxf(st.m, top_z) : st.m;
        const Exponent whole(reference(top), c);
        float shrink = 1.0f; // from their maximum to the row's
        double rest = 0.0, total = st.s;
        const double outside = st.s;
        if constexpr (Op::kTail) {
            float in = 0.0f;
            for (uint32_t k = t & 63; k < args.K; k += kWave)
                if (l.col[k] >= 0)
                    in += exp2_fast(whole.at(l.z[k]));
            in = wave_reduce<OpSum>(in);
            shrink = exp2_fast(fmaxf(whole.at(st.m), kLowest));
            total = (double)st.s * shrink + (double)in;
            if (listed < V && Q < 1.0)
                rest = 1.0 - Q;
            if (rest <= kRestRounding * (1.0 + fabs((double)r.teacher_lse)) &&
                ((double)st.m - (double)reference(top)) * (double)args.scale < kNoTerm)
                rest = 0.0;
            rest = uniform(rest);
        }
        if (t < kWave) {
            // Lanes 0, 1 and 2 take the three logarithms at once.
            // The columns outside as they are in the row's sum, so that what is
            // off in both falls out of p_r; by logits where that may underflow.
            const bool far = !(shrink > kFar);
            const double ln = log(t == 0   ? total
                                  : t == 1 ? rest
                                           : outside * (far ? 1.0 : (double)shrink));
            const double ln_s = __shfl(ln, 0), ln_rest = __shfl(ln, 1), ln_out = __shfl(ln, 2);
            const double ref = reference(top_z), scale = args.scale, most = reference(top);
            double loss = *l.cross + Q * ((most - ref) * scale + ln_s);
            if (Op::kTail && rest > 0.0)
                loss += rest *
                        (ln_rest - ln_out + ln_s - (far ? ((double)st.m - most) * scale : 0.0));
            if (leader) {
                args.join.put(row, (double)r.weight * loss);
                if (args.row_loss_out)
                    args.row_loss_out[row] = (float)loss;
            }
        }
        factor = r.weight * args.scale;
        mass = (float)(Q + rest);
        // Against the maximum of st: the gradient of the columns outside is
        // p_v (Q + q_r) less their share of q_r, which does not shrink with p_v.
        double a = (Q + rest) * (double)shrink / total;
        if (Op::kTail && outside > 0.0)
            a -= rest / outside;
        slope = {(float)((double)factor * a), 0.0f};
        listed_ref = uniform(whole.ref);
        listed_sum = uniform((float)total);
    } else {
        slope = Op::done(args, r, row, st, zy, leader, fix);
    }
    const unsigned before = t < kWave ? join.arrive(row) : 0;

    if constexpr (GRAD) {
        S* dvec = dr + sp.head;
        write_chunk<T, GT, NV, Op::kEntropy>(v, dvec, (chunks - 1) * kChunk, sp.nvec, t, ex, slope);
        if constexpr (MULTI)
            for (uint32_t ch = chunks - 1; ch-- > 0;) {
                load_chunk<T, GT, NV, true>(vec, ch * kChunk, sp.nvec, t, v);
                write_chunk<T, GT, NV, Op::kEntropy>(v, dvec, ch * kChunk, sp.nvec, t, ex, slope);
            }
        if (has_one)
            dr[at_one] = T::narrow(slope_at<Op::kEntropy>(ex.at(one), slope));
        // The few columns with more to them are written again, after the
        // stores above.
        if constexpr (Op::kList) {
            if constexpr (GT > kWave)
                __syncthreads();
            const Exponent whole(listed_ref, c);
            for (uint32_t k = t; k < args.K; k += GT)
                if (l.col[k] >= 0)
                    dr[l.col[k]] = T::narrow(
                        factor * (exp2_fast(whole.at(l.z[k])) / listed_sum * mass - l.q[k]));
        } else {
            uint32_t owner = 0;
            if (r.y >= sp.head && r.y < sp.tail)
                owner = (r.y - sp.head) / T::W % GT;
            else
                owner = r.y < sp.head ? r.y : r.y - sp.tail + sp.head;
            if (t == owner)
                dr[r.y] = T::narrow(slope_at<Op::kEntropy>(ex.at(zy), slope) + fix);
        }
    }
    if (t < kWave)
        join.finish(before, row, rows);
}

// ---- few long rows ------------------------------------------------------------
//
// One workgroup for a row leaves most of the device idle when rows are few and
// long, so a row is cut into segments of a workgroup each.  A segment's
// statistics go to the workspace, and the workgroup that comes last in its row
// joins them, in the order of the segments, and finishes the row.  (The same
// protocol as for the losses' sum; the counts of the rows follow its counts.)
// A gradient is written by a second kernel, grad_kernel, from the row's slope.
constexpr uint32_t kSplitRows = 128, kSegmentsMost = kWave;
constexpr uint32_t kSegmentVecs = 1024; // 16 KiB: four vectors for each thread
constexpr uint32_t kRowCounts = (1 + kJoinGroups) * kCountStride;
static_assert(kRowCounts + kSplitRows * kCountStride <= kPairCounts, "a count for each row");

struct Split {
    float* part;      // [row][3][kSegmentsMost]: maximum, sum, entropy sum
    RowSlope* slope;  // [row]; null: no gradient
    unsigned* counts; // [row * kCountStride]
};

template <class T, int NV, class Op>
__global__ __launch_bounds__(256) void split_kernel(const typename T::S* z, uint32_t rows,
                                                    uint32_t V, uint32_t segs, uint32_t per,
                                                    size_t ld, float c, Split split,
                                                    typename Op::Args args)
{
    typedef typename T::S S;
    constexpr int GT = 256;
    __shared__ float parts[3 * (GT / kWave)];
    const uint32_t t = threadIdx.x, row = blockIdx.x / segs, seg = blockIdx.x % segs;
    const S* zr = z + (size_t)row * ld;
    const Span sp = Span::of<T>(zr, V);
    const typename Op::Row r = Op::begin(args, row, V);
    auto join = Op::join(args, r);
    if (!r.live) {
        if (seg == 0 && t < kWave) {
            Op::dead(args, row, t == 0);
            if (split.slope && t == 0)
                split.slope[row] = {0.0f, 0.0f, 0.0f, 0.0f};
            join.finish(join.arrive(row), row, rows);
        }
        return;
    }
    const u32x4_t* vec = reinterpret_cast<const u32x4_t*>(zr + sp.head);
    const uint32_t first = seg * per;
    const uint32_t last = first + per < sp.nvec ? first + per : sp.nvec;
    const bool has_one = seg == 0 && t < sp.singles;
    const S raw_one = zr[has_one ? sp.single(t) : 0];
    const S raw_zy = zr[r.y];
    u32x4_t v[NV];
    load_chunk<T, GT, NV, false>(vec, first, last, t, v);
    const float one = has_one ? T::widen(raw_one) : -INFINITY, zy = T::widen(raw_zy);
    Stat st = {-INFINITY, 0.0f, 0.0f};
    fold_chunk<T, GT, NV, Op::kEntropy>(v, first, last, t, one, false, c, TakeAll{}, st);
    for (uint32_t next = first + GT * NV; next < last; next += GT * NV) {
        load_chunk<T, GT, NV, false>(vec, next, last, t, v);
        fold_chunk<T, GT, NV, Op::kEntropy>(v, next, last, t, -INFINITY, true, c, TakeAll{}, st);
    }
    st = combine<GT, Op::kEntropy>(st, c, parts);
    if (t >= kWave)
        return;
    float* mine = split.part + (size_t)row * 3 * kSegmentsMost;
    unsigned before = 0;
    if (t == 0) {
        store_shared(mine + seg, st.m);
        store_shared(mine + kSegmentsMost + seg, st.s);
        if constexpr (Op::kEntropy)
            store_shared(mine + 2 * kSegmentsMost + seg, st.u);
        before = count_shared(split.counts + row * kCountStride);
    }
    if (__builtin_amdgcn_readfirstlane(before) != segs - 1)
        return;
    st = {-INFINITY, 0.0f, 0.0f};
    if (t < segs) {
        st.m = load_shared(mine + t);
        st.s = load_shared(mine + kSegmentsMost + t);
        if constexpr (Op::kEntropy)
            st.u = load_shared(mine + 2 * kSegmentsMost + t);
    }
    st = combine<kWave, Op::kEntropy>(st, c, parts);
    float fix;
    const Slope slope = Op::done(args, r, row, st, zy, t == 0, fix);
    if (t == 0) {
        clear_shared(split.counts + row * kCountStride);
        if (split.slope)
            split.slope[row] = {reference(st.m), slope.a, slope.b, fix};
    }
    join.finish(join.arrive(row), row, rows);
}

// ---- a gradient whose statistics are there already --------------------------
//
// A segment of GT * NV vectors of a row per group of threads: nothing is
// reduced, so rows are cut as finely as the device wants.  One read and one
// write: 4096 rows of 131072 bf16 in 337 us, 6.4 TB/s.

// Gradient of the log-probability (glogp) and the entropy (gentropy):
//   dz = scale (g (delta_vy - p) - h p (ln p + H)),  ln p = scale z - lse.
// p = 2^((z - lse / scale) c): the row's reference is lse / scale.
template <bool ENT>
struct LogprobGradOp {
    static constexpr bool kEntropy = ENT;
    static constexpr int kPieceVecs = 2;
    struct Args {
        const int64_t* targets;
        const float *lse, *entropy, *glogp, *gentropy;
        float scale;
        double inverse; // 1 / scale
    };
    struct Row {
        bool live, hit;
        uint32_t y;
        float ref, fix;
        Slope slope;
    };
    static __device__ __forceinline__ Row begin(const Args& a, size_t row, uint32_t V, float c)
    {
        Row r;
        const int64_t y = a.targets[row];
        r.hit = (uint64_t)y < V;
        r.y = r.hit ? (uint32_t)y : 0u;
        const float g = r.hit ? a.glogp[row] : 0.0f, h = ENT ? a.gentropy[row] : 0.0f;
        r.live = g != 0.0f || h != 0.0f;
        const double ref = (double)a.lse[row] * a.inverse;
        r.ref = (float)ref;
        // p = 2^((z - ref) c); what fp32 drops of ref is one more factor.
        const float lost = fabsf(r.ref) < INFINITY ? (float)((ref - (double)r.ref) * (double)c) : 0.0f;
        const float back = exp2f(-lost) * a.scale;
        r.fix = g * a.scale;
        r.slope = {-back * g, 0.0f};
        if constexpr (ENT) {
            r.slope.a = -back * fmaf(h, a.entropy[row] - lost * (float)kLn2, g);
            r.slope.b = -back * h * (float)kLn2;
        }
        return r;
    }
};

// Second pass of the preference loss: the row's slope times d logp / dz.
struct PreferenceGradOp {
    static constexpr bool kEntropy = false;
    static constexpr int kPieceVecs = 2;
    struct Args {
        const int64_t* targets;
        const float2* stat;
        const float* slope;
    };
    struct Row {
        bool live, hit;
        uint32_t y;
        float ref, fix;
        Slope slope;
    };
    static __device__ __forceinline__ Row begin(const Args& a, size_t row, uint32_t V, float)
    {
        Row r;
        const int64_t y = a.targets[row];
        r.hit = (uint64_t)y < V;
        r.y = r.hit ? (uint32_t)y : 0u;
        const float g = r.hit ? a.slope[row] : 0.0f;
        r.live = g != 0.0f;
        const float2 st = a.stat[row];
        r.ref = reference(st.x);
        r.fix = g;
        r.slope = {-g / st.y, 0.0f};
        return r;
    }
};

// The gradient of a row split over several workgroups.
template <bool ENT>
struct SplitGradOp {
    static constexpr bool kEntropy = ENT;
    static constexpr int kPieceVecs = 4;
    struct Args {
        const int64_t* targets;
        const RowSlope* slope;
    };
    struct Row {
        bool live, hit;
        uint32_t y;
        float ref, fix;
        Slope slope;
    };
    static __device__ __forceinline__ Row begin(const Args& a, size_t row, uint32_t V, float)
    {
        Row r;
        const int64_t y = a.targets[row];
        const RowSlope s = a.slope[row];
        r.hit = (uint64_t)y < V;
        r.y = r.hit ? (uint32_t)y : 0u;
        r.live = s.a != 0.0f || s.b != 0.0f || s.fix != 0.0f;
        r.ref = s.ref;
        r.fix = s.fix;
        r.slope = {s.a, s.b};
        return r;
    }
};

template <class T, int GT, int NV, class Op>
__global__ __launch_bounds__(256) void grad_kernel(const typename T::S* z, typename T::S* dz,
                                                   uint32_t rows, uint32_t V, uint32_t segs,
                                                   size_t ld, size_t ldd, float c,
                                                   typename Op::Args args)
{
    typedef typename T::S S;
    constexpr int kGroups = 256 / GT;
    const uint32_t t = threadIdx.x % GT;
    const uint32_t item = blockIdx.x * kGroups + __builtin_amdgcn_readfirstlane(threadIdx.x / GT);
    const uint32_t row = item / segs, first = (item % segs) * (GT * NV);
    if (row >= rows)
        return;
    const S* zr = z + (size_t)row * ld;
    S* dr = dz + (size_t)row * ldd;
    const Span sp = Span::of<T>(zr, V);
    const typename Op::Row r = Op::begin(args, row, V, c);
    const bool has_one = first == 0 && t < sp.singles;
    const uint32_t at_one = has_one ? sp.single(t) : 0;
    if (!r.live) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = first + k * GT + t;
            if (j < sp.nvec)
                store_vec(dr + sp.head + (size_t)j * T::W, u32x4_t{0, 0, 0, 0});
        }
        if (has_one)
            dr[at_one] = 0;
        return;
    }
    const S raw_one = zr[at_one];
    // The thread that writes the target's column reads it first: in place,
    // another thread's read could come after that write.
    bool mine = false;
    if (r.hit) {
        if (r.y >= sp.head && r.y < sp.tail) {
            const uint32_t j = (r.y - sp.head) / T::W;
            mine = j >= first && j - first < GT * NV && (j - first) % GT == t;
        } else {
            mine = has_one && at_one == r.y;
        }
    }
    const S raw_zy = zr[mine ? r.y : at_one];
    u32x4_t v[NV];
    load_chunk<T, GT, NV, true>(reinterpret_cast<const u32x4_t*>(zr + sp.head), first, sp.nvec, t,
                                v);
    const float one = T::widen(raw_one), zy = T::widen(raw_zy);
    const Exponent ex(r.ref, c);
    write_chunk<T, GT, NV, Op::kEntropy>(v, dr + sp.head, first, sp.nvec, t, ex, r.slope);
    if (has_one)
        dr[at_one] = T::narrow(slope_at<Op::kEntropy>(ex.at(one), r.slope));
    if (mine)
        dr[r.y] = T::narrow(slope_at<Op::kEntropy>(ex.at(zy), r.slope) + r.fix);
}

// ---- launches ----------------------------------------------------------------

struct Part { // rows [row0, row0 + rows) of the `all` of a call, on `stream`
    size_t row0;
    uint32_t rows;
    hipStream_t stream;
    size_t all;
    bool first() const { return row0 == 0; }
    bool last() const { return row0 + rows == all; }
};

inline float exponent_scale(float scale) { return (float)((double)scale * kLog2e); }

template <class T, int GT, int NV, bool MULTI, bool GRAD, class Op>
void launch_rows_as(const Logits& m, const Part& p, const typename Op::Args& args, size_t lds)
{
    typedef typename T::S S;
    constexpr uint32_t per = GT < 256 ? 256 / GT : 1;
    const S* z = static_cast<const S*>(m.z) + p.row0 * m.ld;
    S* dz = GRAD ? static_cast<S*>(m.dz) + p.row0 * m.ldd : nullptr;
    hipLaunchKernelGGL((row_kernel<T, GT, NV, MULTI, GRAD, Op>),
                       dim3((p.rows + per - 1) / per), dim3(GT < 256 ? 256 : GT),
                       lds * per, p.stream, z, dz, p.rows, (uint32_t)m.V, m.ld,
                       m.ldd, exponent_scale(m.scale), args);
}

// Whether the rows of a launch are cut into segments.  us a call, whole rows
// against segments, bf16:
//   log-probability, V = 32768: 1 row 3.6 / 3.6, 128 rows 5.0 / 5.6;
//     49152: 5.3 / 4.1, 64 rows 5.9 / 5.4, 128 rows 6.2 / 6.5;
//     65536: 6.4 / 4.2, 128 rows 7.4 / 7.3; 131072: 12.3 / 10.3 for 128 rows
//     and 14.3 / 15.9 for 256;
//   policy loss and gradient, V = 49152: 1 row 8.6 / 8.3, 64 rows 9.2 / 10.4;
//     65536: 10.0 / 8.5 and 10.6 / 10.7; 131072: 15.6 / 8.6 and 16.6 / 13.7,
//     128 rows 17.8 / 20.6; 262144, which a workgroup cannot hold: 32 / 9.1
//     and, for 128 rows, 41 / 36.
template <class T>
bool split_rows(const Logits& m, size_t rows, bool grad)
{
    const size_t nvec = m.V / T::W;
    const size_t many = grad ? 16385 : 8192;
    return rows <= (nvec >= many ? kSplitRows : kSplitRows / 2) && nvec >= (grad ? 8192 : 6144);
}

// The workspace's last mebibyte (before the groups' sums) holds what split
// rows share.
inline Split split_of(const Workspace& ws, bool grad)
{
    char* base = static_cast<char*>(ws.partials) + ws.partial_bytes - (size_t(1) << 20);
    float* part = reinterpret_cast<float*>(base);
    return {part,
            grad ? reinterpret_cast<RowSlope*>(part + kSplitRows * 3 * kSegmentsMost) : nullptr,
            ws.counters + kRowCounts};
}

template <class T, class Op>
void launch_split(const Logits& m, const Part& p, const typename Op::Args& args, const Split& split)
{
    const uint32_t nvec = (uint32_t)(m.V / T::W);
    uint32_t segs = (nvec + kSegmentVecs - 1) / kSegmentVecs;
    segs = segs < kSegmentsMost ? segs : kSegmentsMost;
    const uint32_t per = ((nvec + segs - 1) / segs + 255) / 256 * 256;
    hipLaunchKernelGGL((split_kernel<T, kSegmentVecs / 256, Op>), dim3(p.rows * segs), dim3(256), 0,
                       p.stream, static_cast<const typename T::S*>(m.z) + p.row0 * m.ld, p.rows,
                       (uint32_t)m.V, segs, per, m.ld, exponent_scale(m.scale), split, args);
}

// The threads and registers of a row by its length.  Without a gradient rows
// pass through a wave or, four vectors at a time, through a workgroup: of 256
// threads, or of 512 where rows are few (log-probability, bf16, us a call for
// 256 and 512 threads: 4096 rows of 8192 13.6 and 16.7, 256 rows of 32768 7.1
// and 5.8, of 131072 20.5 and 14.4; eight vectors at a time and 256 threads:
// 15.9, 6.9 and 17.2).  With one a row stays in
// registers: of the smallest group that holds it, so that several rows share a
// compute unit, or, where there are no more rows than compute units, of 256
// or 1024 threads, which take their row through faster (policy loss, bf16, us
// a call for 256 rows and for 1024 rows: V = 4096: 64 threads 8.2 and 9.1, 256
// threads 7.1 and 9.7; V = 32768: 256 threads 12.4 and 26.5, 1024 threads 10.1
// and 30.4; V = 65536: 512 threads 16.7 and 50, 1024 threads 15.7 and 59).  Slots past the row's
// end cost their loads, so short rows have half the slots (8000 rows of 1900
// bf16, 64 threads: eight vectors 18.8, four 16.1).
template <class T, class Op>
void launch_rows_op(const Logits& m, const Part& p, const typename Op::Args& args, size_t lds,
                    const DeviceInfo& dev)
{
    const size_t nvec = m.V / T::W;
    if (!m.dz) {
        if (nvec <= 64 * 8)
            launch_rows_as<T, 64, 8, false, false, Op>(m, p, args, lds);
        else if (nvec >= 4096 && p.rows <= 2u * (uint32_t)dev.cus)
            launch_rows_as<T, 512, 4, true, false, Op>(m, p, args, lds);
        else
            launch_rows_as<T, 256, 4, true, false, Op>(m, p, args, lds);
    } else if constexpr (Op::kHasGrad) {
        const bool few = p.rows <= (uint32_t)dev.cus;
        if (nvec <= 64 * 4)
            launch_rows_as<T, 64, 4, false, true, Op>(m, p, args, lds);
        else if (!few && nvec <= 64 * 8)
            launch_rows_as<T, 64, 8, false, true, Op>(m, p, args, lds);
        else if (nvec <= 256 * 4)
            launch_rows_as<T, 256, 4, false, true, Op>(m, p, args, lds);
        else if (few && nvec <= 1024 * 4)
            launch_rows_as<T, 1024, 4, false, true, Op>(m, p, args, lds);
        else if (nvec <= 256 * 8)
            launch_rows_as<T, 256, 8, false, true, Op>(m, p, args, lds);
        else if (nvec <= 256 * 16)
            launch_rows_as<T, 256, 16, false, true, Op>(m, p, args, lds);
        else if (few && nvec <= 1024 * 8)
            launch_rows_as<T, 1024, 8, false, true, Op>(m, p, args, lds);
        else if (nvec <= 512 * 16)
            launch_rows_as<T, 512, 16, false, true, Op>(m, p, args, lds);
        else if (nvec <= 1024 * 16)
            launch_rows_as<T, 1024, 16, false, true, Op>(m, p, args, lds);
        else
            launch_rows_as<T, 512, 32, true, true, Op>(m, p, args, lds);
    }
}

template <class F>
hipError_t each_part(size_t rows, size_t most, hipStream_t stream, F f)
{
    for (size_t row0 = 0; row0 < rows; row0 += most) {
        const size_t n = rows - row0 < most ? rows - row0 : most;
        f(Part{row0, (uint32_t)n, stream, rows});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// Vectors per thread of the gradient kernel: four where a row fits a
// workgroup so, two in the pieces of a longer one (kernel times of one run, us
// for 4096 rows, four and two: bf16, V = 6598 21.0 and 23.0, 9802 35.4 and 29.4, 131072 348 and 334;
// f32, 131072 725 and 701; eight lose at 20000, 56 and 74).  Of few rows, whose
// slopes a kernel before has left, four (64 rows of 131072 bf16, policy loss:
// 13.7 and 15.2).
constexpr int kGradVecs = 4;

// Workgroups per row of the gradient kernel; 0: several rows per workgroup.
template <class T, class Op>
uint32_t grad_segments(const Logits& m)
{
    const size_t nvec = (m.V + T::W - 1) / T::W, per = 256 * Op::kPieceVecs;
    if (nvec <= 64 * kGradVecs)
        return 0;
    return nvec <= 256 * kGradVecs ? 1 : (uint32_t)((nvec + per - 1) / per);
}

// Rows of one launch of the gradient kernel: at most 2^32 - 1 work-items.
template <class T, class Op>
size_t grad_rows_per_launch(const Logits& m)
{
    const size_t segs = grad_segments<T, Op>(m) ? grad_segments<T, Op>(m) : 1;
    const size_t fit = ((size_t(1) << 24) - 1) / segs;
    return fit < kRowsPerLaunch ? fit : kRowsPerLaunch;
}

// The gradient of rows [row0, row0 + rows), in as many launches as that takes;
// args_from(row) gives the operator's arguments from a row on.
template <class T, class Op, class ArgsFrom>
hipError_t launch_grad(const Logits& m, size_t row0, size_t rows, hipStream_t stream,
                       ArgsFrom args_from)
{
    typedef typename T::S S;
    const float c = exponent_scale(m.scale);
    const uint32_t segs = grad_segments<T, Op>(m);
    return each_part(rows, grad_rows_per_launch<T, Op>(m), stream, [&](const Part& p) {
        const size_t row = row0 + p.row0;
        const S* z = static_cast<const S*>(m.z) + row * m.ld;
        S* dz = static_cast<S*>(m.dz) + row * m.ldd;
        const typename Op::Args args = args_from(row);
        if (!segs)
            hipLaunchKernelGGL((grad_kernel<T, 64, kGradVecs, Op>), dim3((p.rows + 3) / 4),
                               dim3(256), 0, stream, z, dz, p.rows, (uint32_t)m.V, 1u, m.ld, m.ldd,
                               c, args);
        else if (segs == 1)
            hipLaunchKernelGGL((grad_kernel<T, 256, kGradVecs, Op>), dim3(p.rows), dim3(256), 0,
                               stream, z, dz, p.rows, (uint32_t)m.V, segs, m.ld, m.ldd, c, args);
        else
            hipLaunchKernelGGL((grad_kernel<T, 256, Op::kPieceVecs, Op>), dim3(p.rows * segs),
                               dim3(256), 0, stream, z, dz, p.rows, (uint32_t)m.V, segs, m.ld,
                               m.ldd, c, args);
    });
}

} // namespace rowloss

// ---- the calls of one element type -------------------------------------------

template <class T>
bool RowLoss<T>::logprob_shares(const Logits& m)
{
    return rowloss::split_rows<T>(m, m.rows, false);
}

template <class T>
hipError_t RowLoss<T>::logprob(const LogprobCall& a, const DeviceInfo& dev, const Workspace& ws,
                               hipStream_t stream)
{
    using namespace rowloss;
    return each_part(a.m.rows, kRowsPerLaunch, stream, [&](const Part& p) {
        const size_t r = p.row0;
        auto launch = [&](auto op) {
            typedef decltype(op) Op;
            const typename Op::Args args = {a.targets + r, a.logp + r, a.lse + r,
                                            a.entropy ? a.entropy + r : nullptr, a.m.scale};
            if (logprob_shares(a.m))
                launch_split<T, Op>(a.m, p, args, split_of(ws, false));
            else
                launch_rows_op<T, Op>(a.m, p, args, 0, dev);
        };
        if (a.entropy)
            launch(LogprobOp<true>{});
        else
            launch(LogprobOp<false>{});
    });
}

template <class T>
hipError_t RowLoss<T>::logprob_grad(const LogprobGradCall& a, const DeviceInfo&,
                                    hipStream_t stream)
{
    using namespace rowloss;
    auto launch = [&](auto op) {
        typedef decltype(op) Op;
        return launch_grad<T, Op>(a.m, 0, a.m.rows, stream, [&](size_t r) {
            return typename Op::Args{a.targets + r, a.lse + r,
                                     a.gentropy ? a.entropy + r : nullptr, a.glogp + r,
                                     a.gentropy ? a.gentropy + r : nullptr, a.m.scale,
                                     1.0 / (double)a.m.scale};
        });
    };
    return a.gentropy ? launch(LogprobGradOp<true>{}) : launch(LogprobGradOp<false>{});
}

template <class T>
hipError_t RowLoss<T>::distill(const DistillCall& a, const DeviceInfo& dev, const Workspace& ws,
                               hipStream_t stream)
{
    using namespace rowloss;
    const size_t lds = TeacherLds::bytes(bitmap_words((uint32_t)a.m.V), a.K);
    const float mean = (float)(1.0 / (double)a.m.rows);
    hipError_t e = hipSuccess;
    const hipError_t f = each_part(a.m.rows, kRowsPerLaunch, stream, [&](const Part& p) {
        const size_t r = p.row0;
        const Join join = join_of(ws, ws.partials, p.all, a.loss, a.accum);
        const float* weight = a.weight ? a.weight + r : nullptr;
        float* out = a.row_loss ? a.row_loss + r : nullptr;
        const int64_t* idx = a.idx + r * a.ldk;
        const float* val = a.val + r * a.ldk;
        if (a.teacher_lse)
            launch_rows_op<T, DistillOp<true>>(a.m, p,
                                               {idx, val, a.teacher_lse + r, weight, (uint32_t)a.K,
                                                a.ldk, a.m.scale, mean, out, join},
                                               lds, dev);
        else
            launch_rows_op<T, DistillOp<false>>(a.m, p,
                                                {idx, val, nullptr, weight, (uint32_t)a.K, a.ldk,
                                                 a.m.scale, mean, out, join},
                                                lds, dev);
        const hipError_t s = sum_joined(join, p.rows, stream, p.first(), p.last());
        e = e == hipSuccess ? s : e;
    });
    return f == hipSuccess ? e : f;
}

template <class T>
hipError_t RowLoss<T>::policy(const PolicyCall& a, const DeviceInfo& dev, const Workspace& ws,
                              hipStream_t stream)
{
    using namespace rowloss;
    const float mean = (float)(1.0 / (double)a.m.rows);
    hipError_t e = hipSuccess;
    const hipError_t f = each_part(a.m.rows, kRowsPerLaunch, stream, [&](const Part& p) {
        const size_t r = p.row0;
        const Join join = join_of(ws, ws.partials, p.all, a.loss, a.accum);
        auto launch = [&](auto op) {
            typedef decltype(op) Op;
            const typename Op::Args args = {
                a.targets + r, a.old_logp + r, a.ref_logp ? a.ref_logp + r : nullptr,
                a.advantage + r, a.weight ? a.weight + r : nullptr, 1.0 - (double)a.clip_low,
                1.0 + (double)a.clip_high, (double)a.kl_coef, (double)a.entropy_coef, a.m.scale,
                mean, a.logp + r, a.entropy ? a.entropy + r : nullptr, join};
            if (!split_rows<T>(a.m, p.rows, a.m.dz != nullptr))
                return launch_rows_op<T, Op>(a.m, p, args, 0, dev);
            const Split split = split_of(ws, a.m.dz != nullptr);
            launch_split<T, Op>(a.m, p, args, split);
            e = e == hipSuccess ? hipGetLastError() : e;
            if (e != hipSuccess || !a.m.dz)
                return;
            typedef SplitGradOp<Op::kEntropy> GradOp;
            e = launch_grad<T, GradOp>(a.m, r, p.rows, stream, [&](size_t row) {
                return typename GradOp::Args{a.targets + row, split.slope + (row - r)};
            });
        };
        if (a.entropy || a.entropy_coef != 0.0f)
            launch(PolicyOp<true>{});
        else
            launch(PolicyOp<false>{});
        const hipError_t s = sum_joined(join, p.rows, stream, p.first(), p.last());
        e = e == hipSuccess ? s : e;
    });
    return f == hipSuccess ? e : f;
}

template <class T>
hipError_t RowLoss<T>::preference(const PreferenceCall& a, const DeviceInfo& dev, const Workspace& ws,
                                  hipStream_t stream)
{
    using namespace rowloss;
    // Workspace: fp64 log-probabilities, (maximum, sum), slopes, pair losses.
    double* logp = static_cast<double*>(ws.partials);
    float2* stat = reinterpret_cast<float2*>(logp + kPrefRowsMax);
    double* pair_loss = reinterpret_cast<double*>(stat + kPrefRowsMax);
    float* slope = reinterpret_cast<float*>(pair_loss + kPrefPairsMax);
    static_assert(kPrefRowsMax * (8 + 8 + 4) + kPrefPairsMax * 8 <= (size_t(15) << 20),
                  "the statistics fit the workspace, below what split rows share");
    Logits read = a.m;
    read.dz = nullptr;
    // Few rows: many would queue at the pairs' counts and miss the registers
    // that the pairs take (us a call with a kernel for the pairs and without, 2
    // pairs, bf16: 4 rows of 1000 10.3 and 9.0, 64 of 32768 14.3 and 13.0, 256
    // 19.4 and 18.9, 1024 of 1000 12.1 and 17.0).
    const bool joined = a.pairs <= kJoinedPairs && a.m.rows <= (size_t)dev.cus;
    const PairArgs pair = {logp, slope, a.targets, a.starts, a.ref_logp, a.weight, a.seq_logp,
                           join_of(ws, pair_loss, a.pairs, a.loss, a.accum), (int64_t)a.m.rows,
                           (int64_t)a.m.V, (uint32_t)a.pairs, a.kind, a.average, a.beta, a.margin,
                           a.smoothing, ws.counters + kPairCounts};
    // One part: there are at most kPrefRowsMax rows.
    static_assert(kPrefRowsMax <= kRowsPerLaunch, "a row's number is its place in the launch");
    const Part all = {0, (uint32_t)a.m.rows, stream, a.m.rows};
    auto launch = [&](auto op) {
        typedef decltype(op) Op;
        if (split_rows<T>(read, a.m.rows, false))
            launch_split<T, Op>(read, all, {stat, pair}, split_of(ws, false));
        else
            launch_rows_op<T, Op>(read, all, {stat, pair}, 0, dev);
    };
    if (joined)
        launch(PreferenceOp<true>{});
    else
        launch(PreferenceOp<false>{});
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && !joined)
        e = launch_preference_pairs(pair, stream);
    if (e == hipSuccess && a.m.dz)
        e = launch_grad<T, PreferenceGradOp>(a.m, 0, a.m.rows, stream, [&](size_t r) {
            return PreferenceGradOp::Args{a.targets + r, stat + r, slope + r};
        });
    return e;
}

} // namespace red
