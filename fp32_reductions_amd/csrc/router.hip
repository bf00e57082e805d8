// router.hip -- the balance loss of a router of experts, its counts and its
// gradient.
//
//     p = softmax(z_r),  P_e = sum_r w_r p_re,  n_e: how often the rows that
//     count chose expert e,  f = n / sum n
//     loss = b E sum_e f_e P_e + c sum_r w_r lse_r^2
//     dz_r = w_r p_r (q - sum_e p_re q_e + 2 c lse_r),  q = b E f
//
// A row is short (its experts), and the rows are many: 4, 16 or 64 lanes share
// one, and a lane keeps the column sums of its experts in fp32 registers over the
// rows that it takes, 256 at most: more rows go in several launches of the first
// kernel, whose sums are added in fp64.  Counts are integer atomics in LDS, whose order
// changes nothing.  The gradient needs every row's counts, so there are two kernels: the
// sums of each workgroup's rows, which the last of 16 workgroups to arrive adds
// up for its team, and the gradient, whose workgroups each add up the teams (a
// few KB), and which reads the logits again, from a cache in most sizes, and takes
// each row's softmax anew (kept, it would cost as many bytes).  A kernel of its
// own between the two, of one workgroup, took 13.6 of 44 us (65536 x 128 f32).
// Where one workgroup holds all rows at once there is one kernel.
//
// What bounds it is two chains of latencies, each with one read of the logits: 65536 x
// 128 f32 27.0 us (69 MB, 10.6 at 6.5 TB/s), 16384 x 61 bf16 14.6; the one kernel's single
// chain: 96 x 8 bf16 5.3, and 14.7 with two kernels.
//
// The arrivals rest on what gfx950 does with device-scope stores and counts; see
// rowloss_join.hpp.
#include <algorithm>

#include "elements.hpp"
#include "router.hpp"
#include "rowloss_join.hpp"

namespace red {
namespace {

constexpr int kThreads = 1024; // a workgroup of the sums and of the gradient
constexpr double kLog2e64 = 1.4426950408889634074;
constexpr float kLn2f = 0.6931471805599453f;

// Workgroups whose sums one of them adds up, and the most teams of them.
constexpr uint32_t kTeam = 16, kTeams = 32;

// Rows that a lane adds up in fp32.  (4194304 x 256 f32, 4 launches: 2866 us, 2835 in one;
// 1048576 are one launch.)
constexpr uint32_t kRun = 256;
static_assert(kTeams * kCountStride <= kCounterWords, "a count for each team");

struct RouterArgs {
    RouterCall c;
    float* prob_part;               // groups x E
    unsigned* count_part;           // groups x E
    double* z_part;                 // groups
    double* team_prob;              // teams x E
    unsigned long long* team_count; // teams x E
    double* team_z;                 // teams
    unsigned* arrivals;             // of each team's workgroups
    uint32_t groups;
    size_t first, end; // rows of a launch of the sums
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
    // The row's vectors as they are in memory; past its end, anything.
    __device__ __forceinline__ void load(const typename T::S* p, u32x4_t (&v)[NV]) const
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = k * GT + t;
            if (j < nvec) {
                const u32x4u_t u = reinterpret_cast<const u32x4u_t*>(p)[j];
                v[k] = u32x4_t{u.x, u.y, u.z, u.w};
            } else if (rest && j == nvec) {
                v[k] = load_rest<T>(p + (size_t)nvec * W, rest, nvec > 0);
            }
        }
    }
    // Its elements, -inf past its end.
    __device__ __forceinline__ void unpack(const u32x4_t (&v)[NV], float (&f)[NV][W]) const
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = k * GT + t;
            const int here = j < nvec ? W : j == nvec ? (int)rest : 0;
            T::unpack(v[k], f[k]);
#pragma unroll
            for (int i = 0; i < W; ++i)
                f[k][i] = i < here ? f[k][i] : -INFINITY;
        }
    }
    __device__ __forceinline__ void store(typename T::S* p, const float (&f)[NV][W]) const
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t j = k * GT + t;
            const u32x4_t v = T::pack(f[k]);
            if (j < nvec)
                reinterpret_cast<u32x4u_t*>(p)[j] = u32x4u_t{v.x, v.y, v.z, v.w};
            else if (rest && j == nvec)
                store_rest<T>(p + (size_t)nvec * W, v, rest);
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

// What a workgroup keeps in LDS: its counts, and each wave's column sums.
template <class T>
struct RouterLds {
    unsigned* count; // E
    float* prob;     // waves x E
    static size_t bytes(size_t E, int waves) { return E * 4 * (1 + waves); }
    __device__ __forceinline__ RouterLds(unsigned* lds, uint32_t E)
        : count(lds), prob(reinterpret_cast<float*>(lds + E))
    {
    }
};

// A row's choices into the counts; `first` is this lane's first, loaded before.
__device__ __forceinline__ int64_t first_choice(const RouterCall& c, size_t r, uint32_t t)
{
    return t < c.K ? c.experts[r * c.ldk + t] : -1;
}
template <int GT>
__device__ __forceinline__ void count_choices(const RouterCall& c, size_t r, uint32_t t,
                                              int64_t first, unsigned* count)
{
    for (uint32_t k = t; k < c.K; k += GT) {
        const int64_t e = k == t ? first : c.experts[r * c.ldk + k];
        if (e >= 0 && e < (int64_t)c.m.V)
            atomicAdd(&count[e], 1u);
    }
}

// The column sums of a wave's lanes that own the same experts, to LDS.
template <int GT, int NV, int W>
__device__ __forceinline__ void put_columns(float (&acc)[NV][W], uint32_t t, uint32_t E, float* prob)
{
    const uint32_t lane = threadIdx.x % kWave;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) {
#pragma unroll
            for (int d = GT; d < kWave; d *= 2)
                acc[k][i] += __shfl_xor(acc[k][i], d);
            const uint32_t e = (k * GT + t) * W + i;
            if (lane < GT && e < E)
                prob[threadIdx.x / kWave * E + e] = acc[k][i];
        }
}

// Step one, by every workgroup: the sums of its rows, to the workspace, where
// the last of kTeam workgroups to arrive adds up the team's, in order.
template <class T, int GT, int NV>
__global__ __launch_bounds__(kThreads) void router_sum_kernel(RouterArgs a)
{
    extern __shared__ unsigned lds[];
    constexpr int W = T::W, RB = kThreads / GT, WAVES = kThreads / kWave;
    const RouterCall& c = a.c;
    const uint32_t E = (uint32_t)c.m.V;
    const RouterLds<T> mine(lds, E);
    const RouterRow<T, GT, NV> at(E);
    __shared__ double lds_z[WAVES];
    __shared__ unsigned lds_before;
    for (uint32_t e = threadIdx.x; e < E; e += kThreads)
        mine.count[e] = 0;
    __syncthreads();
    float acc[NV][W] = {};
    double zsum = 0.0;
    const size_t step = (size_t)a.groups * RB;
    const bool more = a.first > 0; // added to the launches' before
    // The next row is requested before this one is worked on (not where a row takes
    // a quarter of the registers).
    constexpr bool kAhead = NV < 8;
    size_t r = a.first + (size_t)blockIdx.x * RB + threadIdx.x / GT;
    u32x4_t next[NV] = {};
    float wn = 0.0f;
    int64_t en = -1;
    const auto request = [&](size_t row) {
        wn = row_weight(c, row);
        en = first_choice(c, row, at.t);
        at.load(static_cast<const typename T::S*>(c.m.z) + row * c.m.ld, next);
    };
    if (kAhead && r < a.end)
        request(r);
    for (; r < a.end; r += step) {
        if (!kAhead)
            request(r);
        u32x4_t v[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k)
            v[k] = next[k];
        const float w = wn;
        const int64_t chosen = en;
        if (kAhead && r + step < a.end)
            request(r + step);
        if (w == 0.0f)
            continue;
        float f[NV][W], m, s;
        count_choices<GT>(c, r, at.t, chosen, mine.count);
        at.unpack(v, f);
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
    put_columns<GT>(acc, at.t, E, mine.prob);
    zsum = wave_sum64(zsum);
    if (threadIdx.x % kWave == 0)
        lds_z[threadIdx.x / kWave] = zsum;
    __syncthreads();
    const uint32_t g = blockIdx.x;
    for (uint32_t e = threadIdx.x; e < E; e += kThreads) {
        float p = 0.0f;
#pragma unroll
        for (int k = 0; k < WAVES; ++k)
            p += mine.prob[k * E + e];
        store_shared(a.prob_part + (size_t)g * E + e, p);
        store_shared(reinterpret_cast<float*>(a.count_part + (size_t)g * E + e),
                     __uint_as_float(mine.count[e]));
    }
    if (threadIdx.x == 0) {
        double v = 0.0;
        for (int k = 0; k < WAVES; ++k)
            v += lds_z[k];
        store_shared(a.z_part + g, v);
    }
    // Every thread's stores have arrived before its workgroup is counted.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const uint32_t team = g / kTeam, first = team * kTeam;
    const uint32_t size = a.groups - first < kTeam ? a.groups - first : kTeam;
    unsigned* count = a.arrivals + team * kCountStride;
    if (threadIdx.x == 0)
        lds_before = count_shared(count);
    __syncthreads();
    if (lds_before != size - 1)
        return;
    if (threadIdx.x == 0)
        clear_shared(count);
    for (uint32_t e = threadIdx.x; e < E; e += kThreads) {
        double sum = 0.0;
        unsigned long long chosen = 0;
        constexpr uint32_t kAtOnce = 8;
        for (uint32_t from = 0; from < size; from += kAtOnce) {
            float p[kAtOnce];
            unsigned n[kAtOnce];
#pragma unroll
            for (uint32_t k = 0; k < kAtOnce; ++k) {
                const size_t i = (size_t)(first + (from + k < size ? from + k : 0)) * E + e;
                p[k] = load_shared(a.prob_part + i);
                n[k] = __float_as_uint(load_shared(reinterpret_cast<const float*>(a.count_part + i)));
            }
#pragma unroll
            for (uint32_t k = 0; k < kAtOnce; ++k) {
                sum += from + k < size ? (double)p[k] : 0.0;
                chosen += from + k < size ? n[k] : 0;
            }
        }
        const size_t at_team = (size_t)team * E + e;
        a.team_prob[at_team] = more ? a.team_prob[at_team] + sum : sum;
        a.team_count[at_team] = more ? a.team_count[at_team] + chosen : chosen;
    }
    if (threadIdx.x == 0) {
        double v = 0.0;
        for (uint32_t k = 0; k < size; ++k)
            v += load_shared(a.z_part + first + k);
        a.team_z[team] = more ? a.team_z[team] + v : v;
    }
}

__device__ __forceinline__ unsigned long long block_total(unsigned long long v, unsigned long long* lds)
{
    for (int d = 1; d < kWave; d *= 2)
        v += __shfl_xor(v, d);
    if (threadIdx.x % kWave == 0)
        lds[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0;
    for (uint32_t k = 0; k < blockDim.x / kWave; ++k)
        v += lds[k];
    return v;
}
__device__ __forceinline__ double block_total(double v, double* lds)
{
    v = wave_sum64(v);
    if (threadIdx.x % kWave == 0)
        lds[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0;
    for (uint32_t k = 0; k < blockDim.x / kWave; ++k)
        v += lds[k];
    return v;
}

// Experts of a thread that joins, kThreads apart.
constexpr int kJoined = (int)(kRouterExpertsMax / kThreads);

// The factors q from the counts n of thread's experts, to LDS; where `tell`, the
// outputs too, from the probabilities and the threads' parts z of the sum of
// w lse^2.
template <class Prob>
__device__ __forceinline__ void join(const RouterCall& c, const unsigned long long (&n)[kJoined],
                                     bool tell, Prob prob, double z, float* q)
{
    __shared__ unsigned long long lds_n[kThreads / kWave];
    __shared__ double lds_p[kThreads / kWave];
    const uint32_t E = (uint32_t)c.m.V;
    unsigned long long total = 0;
#pragma unroll
    for (int k = 0; k < kJoined; ++k)
        total += n[k];
    total = block_total(total, lds_n);
    const double b = total ? (double)c.balance * (double)E / (double)total : 0.0;
    double part = 0.0;
#pragma unroll
    for (int k = 0; k < kJoined; ++k) {
        const uint32_t e = threadIdx.x + k * kThreads;
        if (e >= E)
            break;
        const double qe = b * (double)n[k];
        q[e] = (float)qe;
        if (tell) {
            const double p = prob(e);
            part += total ? qe * p : 0.0; // without a choice p has no part in the loss
            c.counts[e] = (int64_t)n[k];
            if (c.prob)
                c.prob[e] = (float)p;
        }
    }
    if (tell) {
        part += c.z != 0.0f ? (double)c.z * z : 0.0;
        part = block_total(part, lds_p);
        if (threadIdx.x == 0)
            c.loss[0] = (float)((c.accum ? (double)c.loss[0] : 0.0) + part);
    }
    __syncthreads();
}

// The gradient from a row's exponentials, with the factors q(k, i).
template <int GT, int NV, int W, class Q>
__device__ __forceinline__ void gradient(const RouterCall& c, float (&f)[NV][W], float m, float s,
                                         float w, Q q)
{
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i)
            dot += f[k][i] * q(k, i);
    dot = group_reduce<OpSum, GT>(dot);
    const float inverse = 1.0f / s;
    const float lse = m + __builtin_amdgcn_logf(s) * kLn2f;
    const float offset = 2.0f * c.z * lse - dot * inverse, scale = w * inverse;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i)
            f[k][i] *= scale * (q(k, i) + offset);
}

// Step two: every workgroup adds up the teams' counts; the last one tells the
// outputs, and the others write the gradient of their rows.
template <class T, int GT, int NV>
__global__ __launch_bounds__(kThreads) void router_grad_kernel(RouterArgs a)
{
    extern __shared__ unsigned lds[];
    constexpr int W = T::W, RB = kThreads / GT;
    const RouterCall& c = a.c;
    const uint32_t E = (uint32_t)c.m.V, teams = (a.groups + kTeam - 1) / kTeam;
    const RouterRow<T, GT, NV> at(E);
    float* lds_q = reinterpret_cast<float*>(lds); // GT NV W, zeros past the last expert
    for (uint32_t e = E + threadIdx.x; e < GT * NV * W; e += kThreads)
        lds_q[e] = 0.0f;
    // This workgroup's first rows are on their way meanwhile.
    const bool tells = blockIdx.x + 1 == gridDim.x;
    const size_t step = (size_t)(gridDim.x - 1) * RB;
    size_t r = tells ? c.m.rows : (size_t)blockIdx.x * RB + threadIdx.x / GT;
    u32x4_t v[NV] = {};
    float w = 0.0f;
    const auto request = [&](size_t row) {
        w = row_weight(c, row);
        at.load(static_cast<const typename T::S*>(c.m.z) + row * c.m.ld, v);
    };
    constexpr bool kAhead = NV < 8;
    if (kAhead && r < c.m.rows)
        request(r);
    unsigned long long n[kJoined];
#pragma unroll
    for (int k = 0; k < kJoined; ++k) {
        const uint32_t e = threadIdx.x + k * kThreads;
        n[k] = 0;
        if (e < E)
#pragma unroll 8
            for (uint32_t g = 0; g < teams; ++g)
                n[k] += a.team_count[(size_t)g * E + e];
    }
    double p[kJoined], z = 0.0;
    if (tells) {
        z = threadIdx.x < teams ? a.team_z[threadIdx.x] : 0.0;
#pragma unroll
        for (int k = 0; k < kJoined; ++k) {
            const uint32_t e = threadIdx.x + k * kThreads;
            p[k] = 0.0;
            if (e < E)
#pragma unroll 8
                for (uint32_t g = 0; g < teams; ++g)
                    p[k] += a.team_prob[(size_t)g * E + e];
        }
    }
    join(c, n, tells, [&](uint32_t e) { return p[e / kThreads]; }, z, lds_q);
    if (tells)
        return;
    // The lane's factors stay in registers, or in LDS where a row takes a quarter of
    // those.
    const auto in_lds = [&](int k, int i) { return lds_q[(k * GT + at.t) * W + i]; };
    float q[NV][W];
    if constexpr (kAhead) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i)
                q[k][i] = in_lds(k, i);
    }
    for (; r < c.m.rows; r += step) {
        if (!kAhead)
            request(r);
        float f[NV][W] = {};
        if (w != 0.0f) {
            float m, s;
            at.unpack(v, f);
            exponentials<GT>(f, m, s);
            if constexpr (kAhead)
                gradient<GT>(c, f, m, s, w, [&](int k, int i) { return q[k][i]; });
            else
                gradient<GT>(c, f, m, s, w, in_lds);
        }
        at.store(static_cast<typename T::S*>(c.m.dz) + r * c.m.ldd, f);
        if (kAhead && r + step < c.m.rows)
            request(r + step);
    }
}

// All of it by one workgroup that holds every row in its registers.
template <class T, int GT, int NV>
__global__ __launch_bounds__(kThreads) void router_one_kernel(RouterCall c)
{
    extern __shared__ unsigned lds[];
    constexpr int W = T::W;
    const uint32_t E = (uint32_t)c.m.V, waves = blockDim.x / kWave;
    const RouterLds<T> mine(lds, E);
    const RouterRow<T, GT, NV> at(E);
    const size_t r = threadIdx.x / GT;
    u32x4_t v[NV] = {};
    float w = 0.0f;
    int64_t chosen = -1;
    if (r < c.m.rows) {
        w = row_weight(c, r);
        chosen = first_choice(c, r, at.t);
        at.load(static_cast<const typename T::S*>(c.m.z) + r * c.m.ld, v);
    }
    for (uint32_t e = threadIdx.x; e < E; e += blockDim.x)
        mine.count[e] = 0;
    __syncthreads();
    float f[NV][W] = {}, p[NV][W] = {}, m = 0.0f, s = 0.0f;
    double z = 0.0;
    if (w != 0.0f) {
        count_choices<GT>(c, r, at.t, chosen, mine.count);
        at.unpack(v, f);
        exponentials<GT>(f, m, s);
        const float scale = w / s;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i)
                p[k][i] = f[k][i] * scale;
        if (c.z != 0.0f && at.t == 0) {
            const double lse = m + __builtin_amdgcn_logf(s) * kLn2f;
            z = (double)w * lse * lse;
        }
    }
    put_columns<GT>(p, at.t, E, mine.prob);
    __syncthreads();
    unsigned long long n[kJoined];
    double sum[kJoined];
#pragma unroll
    for (int k = 0; k < kJoined; ++k) {
        const uint32_t e = threadIdx.x + k * kThreads;
        n[k] = e < E ? mine.count[e] : 0;
        sum[k] = 0.0;
        if (e < E)
            for (uint32_t x = 0; x < waves; ++x)
                sum[k] += (double)mine.prob[x * E + e];
    }
    // q goes where this thread's experts had their counts.
    join(c, n, true, [&](uint32_t e) { return sum[e / kThreads]; }, z,
         reinterpret_cast<float*>(mine.count));
    if (!c.m.dz || r >= c.m.rows)
        return;
    if (w != 0.0f) {
        const float* q = reinterpret_cast<const float*>(mine.count);
        gradient<GT>(c, f, m, s, w, [&](int k, int i) {
            const uint32_t e = (k * GT + at.t) * W + i;
            return e < E ? q[e] : 0.0f;
        });
    }
    at.store(static_cast<typename T::S*>(c.m.dz) + r * c.m.ldd, f);
}


template <class T, int GT, int NV>
hipError_t launch(const RouterCall& c, const DeviceInfo& dev, const Workspace& ws, hipStream_t s)
{
    constexpr size_t RB = kThreads / GT;
    const size_t E = c.m.V;
    if (c.m.rows <= RB && E <= kThreads) {
        // As many threads as its rows and its experts need.
        const size_t threads = std::max((c.m.rows * GT + kWave - 1) / kWave * kWave,
                                        (E + kWave - 1) / kWave * kWave);
        hipLaunchKernelGGL((router_one_kernel<T, GT, NV>), dim3(1), dim3((unsigned)threads),
                           RouterLds<T>::bytes(E, (int)(threads / kWave)), s, c);
        return hipGetLastError();
    }
    RouterArgs a = {};
    a.c = c;
    const size_t wanted = (c.m.rows + RB - 1) / RB;
    // The workspace: teams' sums first, then the workgroups'.
    char* p = static_cast<char*>(ws.partials);
    const auto take = [&p](size_t bytes) {
        char* at = p;
        p += (bytes + 255) / 256 * 256;
        return at;
    };
    a.team_prob = reinterpret_cast<double*>(take(sizeof(double) * kTeams * E));
    a.team_count = reinterpret_cast<unsigned long long*>(take(8 * kTeams * E));
    a.team_z = reinterpret_cast<double*>(take(sizeof(double) * kTeams));
    a.z_part = reinterpret_cast<double*>(take(sizeof(double) * kTeams * kTeam));
    const size_t left = ws.partial_bytes - (p - static_cast<char*>(ws.partials)) - 512;
    a.groups = (uint32_t)std::min({wanted, (size_t)dev.cus, (size_t)kTeams * kTeam,
                                   left / (8 * E)});
    a.prob_part = reinterpret_cast<float*>(take(sizeof(float) * a.groups * E));
    a.count_part = reinterpret_cast<unsigned*>(take(sizeof(unsigned) * a.groups * E));
    a.arrivals = ws.counters;
    // One workgroup a compute unit in both kernels (65536 x 128 f32: 27.1 us; two in
    // the sums 32.2, two in the gradient 28.8).
    const size_t most = (size_t)kRun * RB * a.groups;
    for (; a.first < c.m.rows; a.first += most) {
        a.end = std::min(a.first + most, c.m.rows);
        hipLaunchKernelGGL((router_sum_kernel<T, GT, NV>), dim3(a.groups), dim3(kThreads),
                           RouterLds<T>::bytes(E, kThreads / kWave), s, a);
    }
    const size_t groups = 1 + (c.m.dz ? std::min(wanted, (size_t)dev.cus) : 0);
    hipLaunchKernelGGL((router_grad_kernel<T, GT, NV>), dim3((unsigned)groups), dim3(kThreads),
                       sizeof(float) * GT * NV * T::W, s, a);
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
