// linear_ce.hip -- the cross entropy of hidden rows against an output layer and its
// gradients, with no logits of the caller's.
//
//     z = s h W^T,  lse = ln sum_v exp z_v,  row loss = lse - z_t + c lse^2
//     d_v = w s ((1 + 2 c lse) p_v - [v = t]),  dh = d W,  dW = d^T h
//
// The products run on the matrix cores (mfma_tile.hpp).  Forward, a workgroup's
// tile of logits stays in its registers and leaves one maximum and one sum of
// exponentials for each of its rows, which a second kernel joins.  The
// gradients need the whole row's sum before the first of them.  So the products are
// kept, in fp32, where the vocabulary is one piece and they take little room; otherwise
// they are computed a second time, a piece of the vocabulary at a time: 8 rows V D
// operations where keeping them takes 6, and a workspace that does not grow with V.
// The piece's d, rounded to the inputs' type, goes to the workspace (it is an operand of
// both further products), dh gathers d W over the pieces in fp32, and the piece's rows of
// dW are finished at once.
//
// Rows that do not count are left out first: the others' hidden rows are copied
// together (rows D elements, nothing beside rows V D), which also keeps a NaN in
// a masked row out of dW, and makes the products' operand aligned and padded.
//
// What is rounded is d without its row's weight: d / (w s) times the mantissa of w over
// the largest weight, so that where all weights are equal the target's element, the
// largest, of a row that is unsure of it is -1, exactly.  The weights' exponents and the
// largest come back later: dh takes them behind its product, in fp32, exactly; for dW,
// whose sum runs over rows, a copy of the hidden rows has the exponents, exactly but for
// values below the type's normal range.  Half precision has no room there, so its rows
// are put in order of groups of 4 exponents: the copy has what is left within a group
// (2^-3 at least: values are off by 2^-22 at most), and dW's sum is scaled, in fp32, from
// one group to the next.  Weights within a factor of 8 are one group.
// In half precision d is 2^4 times larger, which keeps probabilities down to 4e-6 normal
// numbers and overflows where 1 + 2 c lse passes 2000.
//
// Bf16, us a call: 4096 rows (512 masked) against 131072 x 4096 with both gradients 12840,
// bound by the matrix cores' power; 1 row against 32768 x 4096 54, by the reading of the
// layer (46.5 at 5.8 TB/s) and two small launches; 1021 rows (100 masked) against
// 50001 x 2048, the loss alone, 211.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "linear_ce.hpp"
#include "mfma_tile.hpp"
#include "rowloss_join.hpp"

namespace red {
namespace {

constexpr float kLog2ef = 1.4426950408889634f;
constexpr double kLog2e64 = 1.4426950408889634074;
constexpr float kHalfScale = 16.0f; // of d in half precision

typedef TileShape<256, 256, 2, 4, 64, 2> BigTile;
typedef TileShape<256, 128, 2, 4, 64, 2> HalfTile;   // the last big tiles, cut along n
typedef TileShape<256, 64, 4, 2, 64, 2> QuarterTile;
typedef TileShape<128, 128, 2, 2, 32, 4> MidTile;
typedef TileShape<128, 128, 2, 2, 32, 2> MidWeight;
typedef TileShape<128, 32, 4, 1, 128, 3> FewTile;

// The hidden rows are padded with zeros to multiples of these.
constexpr uint32_t kRowPad = 64, kWidthPad = 64;

// Exponents of a weight over the largest (share_of), in groups: the first has the largest.
constexpr int kExponentMin = -100, kGroupExponents = 4;
constexpr uint32_t kGroups = -kExponentMin / kGroupExponents + 1;
static_assert(kGroups <= kWave, "a lane for each");

// A number that may be past fp32's range, where a product with it need not be.
struct Factor {
    float mantissa;
    int exponent;
    // The exact step first: the other one is one with the rounding to f16.
    __device__ __forceinline__ float times(float v) const { return ldexpf(v, exponent) * mantissa; }
};

// What the kernels share.  Pointers into the workspace, except those of the call.
struct Lce {
    LinearCall c;
    // [0]: rows that count; [1]: the largest of their weights' finite magnitudes (float);
    // [2]: arrivals
    uint32_t* count;
    uint32_t* group;   // half precision's dW: rows of each group of weights
    int32_t* where;    // of each row of the call: its place among those that count, or -1
    int32_t *row, *target; // of each row that counts: its number, its target
    // Weight, target's product, largest product, log2 of the sum of 2^((z - m) scale log2 e),
    // factors of d.
    float *w, *zt, *m, *ls, *fa, *fb;
    Factor* fs; // of dh
    double* loss_part; // of each workgroup that joins rows
    char *h, *hs;      // hidden rows, and a copy times 2^(exponent of their weight)
    size_t ldh;        // bytes
    float2* stat;      // maximum and sum of each row and vocabulary tile
    uint32_t tiles_v;
    float* z;          // kept products, rows x piece
    char* d;           // rows x piece
    uint32_t piece;
    float* dh;         // splits x padded rows x padded width, in tile order
    uint32_t splits, cus;
};

__device__ __forceinline__ uint32_t round_up32(uint32_t v, uint32_t to) { return (v + to - 1) / to * to; }

// ---- rows that count --------------------------------------------------------

__device__ __forceinline__ float weight_of(const LinearCall& c, size_t r)
{
    return c.row_weight ? c.row_weight[r] : 1.0f / (float)c.rows;
}
__device__ __forceinline__ bool counted(const LinearCall& c, size_t r)
{
    const int64_t t = c.targets[r];
    return weight_of(c, r) != 0.0f && t >= 0 && t < (int64_t)c.V;
}

// What the largest is taken of: no infinity or NaN, which would be every row's factor.
__device__ __forceinline__ float magnitude(float w)
{
    const float m = fabsf(w);
    return m < INFINITY ? m : 0.0f;
}

// A weight over the largest: mantissa, 1 to 2 in magnitude, and exponent, 0 or less.
__device__ __forceinline__ Factor share_of(float w, float largest)
{
    const float r = w / largest;
    int e = fabsf(r) > 0.0f && fabsf(r) <= 1.0f ? ilogbf(r) : 0; // 0 where one is no number
    e = e < kExponentMin ? kExponentMin : e;
    return {ldexpf(r, -e), e};
}
// What d is multiplied by behind its products, beside its row's share.
template <class T>
__device__ __forceinline__ Factor factor_of(float largest, float scale)
{
    constexpr double kUp = __is_same(T, ElemF16) ? kHalfScale : 1.0;
    int e;
    const double m = frexp((double)largest * (double)scale / kUp, &e);
    return {(float)(2.0 * m), e - 1};
}
template <bool GROUPED>
__device__ __forceinline__ uint32_t group_of(float w, float largest)
{
    return GROUPED ? (uint32_t)-share_of(w, largest).exponent / kGroupExponents : 0;
}

// The places of the rows that count: in the order of their groups, and of the call
// within one.  One workgroup.
template <bool GROUPED>
__global__ __launch_bounds__(1024) void lce_rows_kernel(Lce a)
{
    constexpr uint32_t kThreads = 1024, kAll = kThreads / kWave, kOf = GROUPED ? kGroups : 1;
    // Each wave's rows of each group and the groups' next places, twice: a turn's are read
    // while the next one's are written.
    __shared__ uint32_t lds[2][kAll][kOf], lds_first[2][kOf + 1];
    __shared__ float lds_w[kAll];
    float largest = 0.0f;
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const auto share_largest = [&] {
        largest = wave_reduce<OpMax>(largest);
        if (lane == 0)
            lds_w[wave] = largest;
        __syncthreads();
        for (uint32_t k = 0; k < kAll; ++k)
            largest = fmaxf(largest, lds_w[k]);
    };
    if (threadIdx.x <= kOf)
        lds_first[0][threadIdx.x] = 0;
    if constexpr (GROUPED) {
        for (size_t r = threadIdx.x; r < a.c.rows; r += kThreads)
            if (counted(a.c, r))
                largest = fmaxf(largest, magnitude(weight_of(a.c, r)));
        share_largest();
        // Each group's rows, at the place of the one before it: then their sums.
        for (size_t r = threadIdx.x; r < a.c.rows; r += kThreads)
            if (counted(a.c, r))
                atomicAdd(&lds_first[0][group_of<true>(weight_of(a.c, r), largest) + 1], 1u);
        __syncthreads();
        if (threadIdx.x < kOf)
            a.group[threadIdx.x] = lds_first[0][threadIdx.x + 1];
        __syncthreads();
        if (threadIdx.x == 0)
            for (uint32_t g = 1; g < kOf; ++g)
                lds_first[0][g] += lds_first[0][g - 1];
    }
    uint32_t turn = 0;
    for (size_t first = 0; first < a.c.rows; first += kThreads, turn ^= 1) {
        const size_t r = first + threadIdx.x;
        const bool counts = r < a.c.rows && counted(a.c, r);
        const float w = counts ? weight_of(a.c, r) : 0.0f;
        const uint32_t g = counts ? group_of<GROUPED>(w, largest) : 0;
        if (lane < kOf)
            lds[turn][wave][lane] = 0;
        __builtin_amdgcn_wave_barrier(); // LDS keeps a wave's order
        uint32_t before = 0; // rows of the group in this wave before this one
        for (uint64_t left = __ballot(counts); left;) {
            const uint32_t of = __builtin_amdgcn_readlane(g, __builtin_ctzll(left));
            const uint64_t same = __ballot(counts && g == of);
            if (g == of)
                before = __popcll(same & ((1ull << lane) - 1));
            if (lane == 0)
                lds[turn][wave][of] = __popcll(same);
            left &= ~same;
        }
        __syncthreads();
        uint32_t at = lds_first[turn][g] + before;
#pragma unroll
        for (uint32_t k = 0; k < kAll; ++k)
            at += k < wave ? lds[turn][k][g] : 0;
        if (r < a.c.rows)
            a.where[r] = counts ? (int32_t)at : -1;
        if (counts) {
            a.row[at] = (int32_t)r;
            a.target[at] = (int32_t)a.c.targets[r];
            a.w[at] = w;
            if (!GROUPED)
                largest = fmaxf(largest, magnitude(w));
        }
        if (threadIdx.x < kOf) {
            uint32_t next = lds_first[turn][threadIdx.x];
#pragma unroll
            for (uint32_t k = 0; k < kAll; ++k)
                next += lds[turn][k][threadIdx.x];
            lds_first[turn ^ 1][threadIdx.x] = next;
        }
    }
    if constexpr (GROUPED)
        __syncthreads();
    else
        share_largest();
    if (threadIdx.x == 0) {
        a.count[0] = lds_first[turn][kOf - 1];
        a.count[1] = __float_as_uint(largest);
        a.count[2] = 0;
    }
}

// Rows up to which lce_gather_kernel goes alone (1024: 18.6 us a call so, 20.2
// otherwise; 2048: 23.7 and 22.4).
constexpr size_t kRowsAlone = 1024;

// One workgroup a row of the call, and kRowPad more for the zeros after the last
// row that counts.  ALONE: there has been no lce_rows_kernel; with few rows each
// workgroup counts those before its own itself, which takes less than a launch.
template <class T, bool ALONE>
__global__ __launch_bounds__(256) void lce_gather_kernel(Lce a)
{
    const size_t r = blockIdx.x;
    const uint32_t D = (uint32_t)a.c.D, chunks = (uint32_t)(a.ldh / 16);
    const bool real = r < a.c.rows;
    const uint16_t* from = static_cast<const uint16_t*>(a.c.hidden) + (real ? r * a.c.ldh : 0);
    // This thread's first chunk of the row is on its way while its place is found.
    // (Past D there are zeros; D is a multiple of 8.)
    const auto chunk = [&](uint32_t i) {
        u32x4_t v = {0, 0, 0, 0};
        if (real && i * 8 < D) {
            const u32x4u_t u = reinterpret_cast<const u32x4u_t*>(from)[i];
            v = u32x4_t{u.x, u.y, u.z, u.w};
        }
        return v;
    };
    const u32x4_t first = chunk(threadIdx.x);
    uint32_t to;
    int32_t at;
    float largest = 0.0f;
    constexpr bool kMayGroup = __is_same(T, ElemF16);
    const bool grouped = kMayGroup && a.hs;
    const auto of_group = [&](float w) { return grouped ? group_of<kMayGroup>(w, largest) : 0; };
    if constexpr (ALONE) {
        __shared__ uint32_t lds[kWaves], lds_group[kGroups];
        __shared__ float lds_w[kWaves];
        constexpr uint32_t kHeld = (uint32_t)kRowsAlone / 256;
        float w[kHeld]; // of rows that count; 0: they do not
#pragma unroll
        for (uint32_t k = 0; k < kHeld; ++k) {
            const uint32_t i = threadIdx.x + k * 256;
            w[k] = i < a.c.rows && counted(a.c, i) ? weight_of(a.c, i) : 0.0f;
            largest = fmaxf(largest, magnitude(w[k]));
        }
        const bool counts = real && counted(a.c, r);
        largest = wave_reduce<OpMax>(largest);
        if (threadIdx.x % kWave == 0)
            lds_w[threadIdx.x / kWave] = largest;
        if (kMayGroup && threadIdx.x < kGroups)
            lds_group[threadIdx.x] = 0;
        __syncthreads();
        largest = fmaxf(fmaxf(lds_w[0], lds_w[1]), fmaxf(lds_w[2], lds_w[3]));
        const uint32_t mine = !real ? kGroups : counts ? of_group(weight_of(a.c, r)) : 0;
        uint32_t n = 0;
#pragma unroll
        for (uint32_t k = 0; k < kHeld; ++k)
            if (w[k] != 0.0f) {
                const uint32_t i = threadIdx.x + k * 256, g = of_group(w[k]);
                n += g < mine || (g == mine && i < r);
                if (!real && grouped)
                    atomicAdd(&lds_group[g], 1u);
            }
        n = (uint32_t)wave_sum64((double)n);
        if (threadIdx.x % kWave == 0)
            lds[threadIdx.x / kWave] = n;
        __syncthreads();
        at = (int32_t)(lds[0] + lds[1] + lds[2] + lds[3]);
        if (threadIdx.x == 0) {
            if (counts) {
                a.row[at] = (int32_t)r;
                a.target[at] = (int32_t)a.c.targets[r];
                a.w[at] = weight_of(a.c, r);
            }
            if (r == a.c.rows) {
                a.count[0] = (uint32_t)at;
                a.count[1] = __float_as_uint(largest);
                a.count[2] = 0;
            }
        }
        if (grouped && r == a.c.rows && threadIdx.x < kGroups)
            a.group[threadIdx.x] = lds_group[threadIdx.x];
        if (real && !counts)
            at = -1;
    } else {
        at = real ? a.where[r] : (int32_t)a.count[0];
        largest = __uint_as_float(a.count[1]);
    }
    if (real) {
        if (at < 0) {
            if (threadIdx.x == 0) {
                if (a.c.logp)
                    a.c.logp[r] = 0.0f;
                if (a.c.lse)
                    a.c.lse[r] = 0.0f;
            }
            if (a.c.dhidden) {
                uint16_t* out = static_cast<uint16_t*>(a.c.dhidden) + r * a.c.lddh;
                for (uint32_t i = threadIdx.x; i < D; i += 256)
                    out[i] = 0;
            }
            return;
        }
        to = (uint32_t)at;
    } else {
        to = (uint32_t)at + (uint32_t)(r - a.c.rows);
        if (to >= round_up32((uint32_t)at, kRowPad))
            return;
    }
    u32x4_t* out = reinterpret_cast<u32x4_t*>(a.h + to * a.ldh);
    u32x4_t* scaled = a.hs ? reinterpret_cast<u32x4_t*>(a.hs + to * a.ldh) : nullptr;
    // The exponent of its weight, or what its group leaves of that.
    int e = 0;
    if (scaled && real) {
        const float w = weight_of(a.c, r);
        e = share_of(w, largest).exponent + (int)of_group(w) * kGroupExponents;
    }
    const auto put = [&](uint32_t i, const u32x4_t& v) {
        out[i] = v;
        if (!scaled)
            return;
        float f[8];
        T::unpack(v, f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            f[k] = ldexpf(f[k], e);
        scaled[i] = e ? T::pack(f) : v;
    };
    if (threadIdx.x < chunks)
        put(threadIdx.x, first);
    for (uint32_t i = threadIdx.x + 256; i < chunks; i += 256)
        put(i, chunk(i));
}

// ---- tiles ------------------------------------------------------------------

// Workgroup `id` of `total`: each XCD takes a run of the order of tiles ...
__device__ __forceinline__ uint32_t in_order(uint32_t id, uint32_t total)
{
    const uint32_t x = id % kXcds, i = id / kXcds, per = total / kXcds, rest = total % kXcds;
    return x * per + (x < rest ? x : rest) + i;
}
// ... in which 8 tiles along m go with every tile along n, so that what one XCD's
// compute units read at a time is few operand rows, from its own L2.
struct TileAt {
    uint32_t m, n;
};
__device__ __forceinline__ TileAt tile_at(uint32_t o, uint32_t tiles_m, uint32_t tiles_n)
{
    const uint32_t group = o / (8 * tiles_n), in = o % (8 * tiles_n);
    const uint32_t left = tiles_m - group * 8, height = left < 8 ? left : 8;
    return {group * 8 + in % height, in / height};
}

// The work of workgroup `id`: f(shape, tile along m, first row n).  Big tiles come a
// compute unit each, so those of the last round, if they are at most half as many as
// the units, are cut in two or four (PARTS) along n and given to as many.  (921 rows
// against 50001 x 2048, 784 tiles on 256 units: 232 us whole, 216 cut; 600 rows with
// their gradient, 1265 and 1242.)
template <class S, uint32_t PARTS = 4, class F>
__device__ __forceinline__ void with_tile(uint32_t id, uint32_t tiles_m, uint32_t tiles_n, uint32_t cus,
                                          F f)
{
    const uint32_t total = tiles_m * tiles_n;
    if constexpr (__is_same(S, BigTile)) {
        const uint32_t rest = total % cus, whole = total - rest;
        const uint32_t parts = PARTS == 4 && rest * 4 <= cus ? 4 : rest * 2 <= cus ? 2 : 1;
        if (id >= whole) {
            const uint32_t k = id - whole;
            if (k >= rest * parts)
                return;
            const TileAt t = tile_at(whole + k / parts, tiles_m, tiles_n);
            const uint32_t n0 = t.n * S::N + k % parts * (S::N / parts);
            if (parts == 1)
                f(S(), t.m, n0);
            else if (parts == 2)
                f(HalfTile(), t.m, n0);
            else if constexpr (PARTS == 4)
                f(QuarterTile(), t.m, n0);
            return;
        }
        const TileAt t = tile_at(in_order(id, whole), tiles_m, tiles_n);
        f(S(), t.m, t.n * S::N);
    } else {
        if (id >= total)
            return;
        const TileAt t = tile_at(in_order(id, total), tiles_m, tiles_n);
        f(S(), t.m, t.n * S::N);
    }
}
// Workgroups enough for that, whatever the rows that count leave of tiles_n.
template <class S>
uint32_t workgroups(uint32_t tiles_m, uint32_t tiles_n, uint32_t cus)
{
    const uint32_t total = tiles_m * tiles_n;
    return total + (__is_same(S, BigTile) ? std::min(cus, total * 3) : 0);
}

__device__ __forceinline__ uint32_t lds_of(char* lds)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
}

// Where a tile of few rows starts along k; the others keep in step, since what they
// read is shared.
template <class S>
__device__ __forceinline__ uint32_t turn_of(uint32_t tile)
{
    return S::N < 256 ? tile * 3 : 0;
}

// ---- forward ------------------------------------------------------------------

// Tile number t along the vocabulary, rows n0 on.
template <class T, class S, bool KEEP>
__device__ __forceinline__ void stat_tile(const Lce& a, char* buffer, uint32_t t, uint32_t n0)
{
    const uint32_t lds = lds_of(buffer), v0 = t * S::M, rows = a.count[0];
    if (n0 >= rows)
        return;
    const Operand W = {static_cast<const char*>(a.c.weight), a.c.ldw * 2, (uint32_t)a.c.V, (uint32_t)a.c.D};
    const Operand H = {a.h, a.ldh, rows, (uint32_t)a.c.D};
    TileAcc<S> acc;
    multiply<T, S, true, true>(acc, W, H, v0, n0, 0, (uint32_t)a.c.D, lds, turn_of<S>(t));

    const float c = a.c.scale * kLog2ef;
    const uint32_t left = (uint32_t)a.c.V - v0; // columns of this tile
    if constexpr (KEEP) {
        // Each wave turns its 32 x 32 blocks in LDS of its own, so that a store writes whole
        // lines of 8 rows, not 32 bytes of 32 (1531 rows against 65537 x 1000: 781 us, 795).
        typedef __attribute__((address_space(3))) f32x4_t* ptr;
        constexpr uint32_t kRow = 32 * 4 + 16; // bytes
        static_assert(S::WM * S::N * 8 + S::kWaves * 32 * kRow <= S::kLds, "behind `part`");
        const uint32_t mine = lds + S::WM * S::N * 8 + threadIdx.x / kWave * (32 * kRow);
        const uint32_t lane = threadIdx.x % kWave;
#pragma unroll
        for (int j = 0; j < S::NS; ++j)
#pragma unroll
            for (int i = 0; i < S::MS; ++i) {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *(ptr)(uintptr_t)(mine + lane % 32 * kRow + (e / 4 * 8 + lane / 32 * 4) * 4) =
                        f32x4_t{acc.c[i][j][e], acc.c[i][j][e + 1], acc.c[i][j][e + 2],
                                acc.c[i][j][e + 3]};
                __builtin_amdgcn_wave_barrier(); // LDS keeps a wave's order
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t r = k * 8 + lane / 8, n = n0 + acc.wave_n() + j * 32 + r;
                    const uint32_t m = acc.wave_m() + i * 32 + lane % 8 * 4;
                    const f32x4_t v = *(ptr)(uintptr_t)(mine + r * kRow + lane % 8 * 16);
                    if (n < rows && m < left) // a.piece is a multiple of 4
                        *reinterpret_cast<f32x4_t*>(a.z + (size_t)n * a.piece + v0 + m) = v;
                }
                __builtin_amdgcn_wave_barrier();
            }
    }
    float2* part = reinterpret_cast<float2*>(buffer); // [WM][N]
#pragma unroll
    for (int j = 0; j < S::NS; ++j) {
        const uint32_t n = acc.n(j);
        if (left < (uint32_t)S::M) {
#pragma unroll
            for (int i = 0; i < S::MS; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (acc.m(i, e) >= left)
                        acc.c[i][j][e] = -INFINITY;
        }
        // The target's product, where it is in this tile.
        const uint32_t at = n0 + n < rows ? (uint32_t)a.target[n0 + n] - v0 : ~0u;
        if (__any(at < (uint32_t)S::M)) {
#pragma unroll
            for (int i = 0; i < S::MS; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (acc.m(i, e) == at)
                        a.zt[n0 + n] = acc.c[i][j][e];
        }
        float m = -INFINITY, s = 0.0f;
#pragma unroll
        for (int i = 0; i < S::MS; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                m = fmaxf(m, acc.c[i][j][e]);
        m = fmaxf(m, __shfl_xor(m, 32));
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < S::MS; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                s += __builtin_amdgcn_exp2f((acc.c[i][j][e] - ref) * c);
        s += __shfl_xor(s, 32);
        if (threadIdx.x % kWave < 32)
            part[threadIdx.x / kWave / S::WN * S::N + n] = make_float2(m, s);
    }
    barrier();
    for (uint32_t n = threadIdx.x; n < (uint32_t)S::N; n += S::kThreads) {
        if (n0 + n >= rows)
            continue;
        float m = -INFINITY, s = 0.0f;
#pragma unroll
        for (int k = 0; k < S::WM; ++k)
            m = fmaxf(m, part[k * S::N + n].x);
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int k = 0; k < S::WM; ++k) {
            const float2 p = part[k * S::N + n];
            s += p.y * __builtin_amdgcn_exp2f((p.x - ref) * c);
        }
        a.stat[(size_t)(n0 + n) * a.tiles_v + t] = make_float2(m, s);
    }
}

__device__ __forceinline__ uint32_t live_tiles(const Lce& a, uint32_t n) { return (a.count[0] + n - 1) / n; }

// `tiles` tiles along the vocabulary, from number `first` on.
template <class T, class S, bool KEEP>
__global__ __launch_bounds__(S::kThreads) void lce_stat_kernel(Lce a, uint32_t first, uint32_t tiles)
{
    __shared__ __align__(1024) char buffer[S::kLds];
    with_tile<S>(blockIdx.x, tiles, live_tiles(a, S::N), a.cus, [&](auto shape, uint32_t m, uint32_t n0) {
        stat_tile<T, decltype(shape), KEEP>(a, buffer, first + m, n0);
    });
}

// One wave a row: its tiles' sums, its loss and the factors of its gradient.  The
// workgroup that arrives last adds up the losses, in order.
constexpr int kJoinThreads = 1024, kJoinWaves = kJoinThreads / kWave;
template <class T>
__device__ __forceinline__ double join_row(const Lce& a, uint32_t n, uint32_t lane)
{
    const float2* stat = a.stat + (size_t)n * a.tiles_v;
    const float c = a.c.scale * kLog2ef;
    // The first 512 tiles stay in registers between the maximum and the sum.
    constexpr uint32_t kHeld = 8;
    const float zt = a.zt[n], weight = a.w[n];
    const uint32_t r = (uint32_t)a.row[n];
    float2 held[kHeld];
    float m = -INFINITY;
#pragma unroll
    for (uint32_t k = 0; k < kHeld; ++k)
        held[k] = lane + k * kWave < a.tiles_v ? stat[lane + k * kWave] : make_float2(-INFINITY, 0.0f);
#pragma unroll
    for (uint32_t k = 0; k < kHeld; ++k)
        m = fmaxf(m, held[k].x);
    for (uint32_t k = lane + kHeld * kWave; k < a.tiles_v; k += kWave)
        m = fmaxf(m, stat[k].x);
    m = wave_reduce<OpMax>(m);
    const float ref = m == -INFINITY ? 0.0f : m;
    double s = 0.0;
#pragma unroll
    for (uint32_t k = 0; k < kHeld; ++k)
        s += (double)(held[k].y * __builtin_amdgcn_exp2f((held[k].x - ref) * c));
    for (uint32_t k = lane + kHeld * kWave; k < a.tiles_v; k += kWave) {
        const float2 p = stat[k];
        s += (double)(p.y * __builtin_amdgcn_exp2f((p.x - ref) * c));
    }
    s = wave_sum64(s);
    if (lane)
        return 0.0;
    const double scale = a.c.scale, w = weight;
    const double ln = log(s), lse = scale * (double)ref + ln;
    const double logp = scale * ((double)zt - (double)ref) - ln;
    if (a.c.logp)
        a.c.logp[r] = (float)logp;
    if (a.c.lse)
        a.c.lse[r] = (float)lse;
    a.m[n] = ref;
    a.ls[n] = (float)(ln * kLog2e64);
    const float largest = __uint_as_float(a.count[1]);
    const Factor share = share_of(weight, largest), f = factor_of<T>(largest, a.c.scale);
    const float up = __is_same(T, ElemF16) ? kHalfScale : 1.0f;
    a.fb[n] = share.mantissa * up;
    a.fa[n] = (float)((double)(share.mantissa * up) * (1.0 + 2.0 * (double)a.c.z * lse));
    a.fs[n] = {f.mantissa, f.exponent + share.exponent};
    return w * ((double)a.c.z * lse * lse - logp);
}

template <class T>
__global__ __launch_bounds__(kJoinThreads) void lce_join_kernel(Lce a)
{
    __shared__ double lds[kJoinWaves];
    __shared__ uint32_t lds_before;
    const uint32_t wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const uint32_t n = blockIdx.x * kJoinWaves + wave;
    const double mine = n < a.count[0] ? join_row<T>(a, n, lane) : 0.0;
    if (lane == 0)
        lds[wave] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        double v = 0.0;
        for (int k = 0; k < kJoinWaves; ++k)
            v += lds[k];
        store_shared(a.loss_part + blockIdx.x, v);
        if (gridDim.x == 1)
            a.c.loss[0] = (float)((a.c.accum ? (double)a.c.loss[0] : 0.0) + v);
        else
            lds_before = count_shared(a.count + 2);
    }
    __syncthreads();
    if (gridDim.x == 1 || lds_before != gridDim.x - 1)
        return;
    double v = 0.0;
    for (uint32_t k = threadIdx.x; k < gridDim.x; k += kJoinThreads)
        v += load_shared(a.loss_part + k);
    v = wave_sum64(v);
    if (lane == 0)
        lds[wave] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = a.c.accum ? (double)a.c.loss[0] : 0.0;
        for (int k = 0; k < kJoinWaves; ++k)
            v += lds[k];
        a.c.loss[0] = (float)v;
    }
}

// ---- a few rows ---------------------------------------------------------------
//
// The layer is only read, so what counts is the rate of its reading: each wave
// takes 16 of its rows from end to end, straight into the operand registers of
// v_mfma_f32_16x16x32 (lane l: row l % 16, 16 bytes at 64 s + 16 (l / 16) in step s),
// with kAhead steps, 128 bytes of each row, in flight twice over (8 steps instead of
// 2: 190.8 us instead of 185.7 for 8 rows against 131072 x 4096); the hidden rows
// stay in LDS (16 bytes of padding a row spread 16 rows over the banks).  Waves start
// at different places of their rows: in step they ask the same few memory channels
// at a time (1 row against 32768 x 4096: 55 us in step, 48 so; tiles through LDS
// took 59).  The blocks that a workgroup's waves would not all have one of are shared,
// a part of k to each wave, whose sums meet in LDS, in order, where that is shorter.
constexpr int kStreamWaves = 8, kStreamThreads = kStreamWaves * kWave, kAhead = 2;
constexpr uint32_t kTurn = 2 * kAhead * 32; // steps of k
constexpr size_t kStreamLds = 156 * 1024;
// More rows take tiles, whose hidden rows need not be in LDS first (32 rows against 32768 x
// 2048: 40.5 us streamed, 35.8 in tiles; 16 rows against 131072 x 2048: 103 and 106).
constexpr size_t kStreamRowsMax = 16;

// LDS for `rows` hidden rows of ldh bytes, and for the waves' sums.
constexpr size_t stream_lds(size_t rows, size_t ldh)
{
    return rows * (ldh + 16) + kStreamWaves * kWave * sizeof(f32x4_t);
}

template <class T>
__device__ __forceinline__ f32x4_t mfma16(const s16x8_t& a, const s16x8_t& b, const f32x4_t& c)
{
    if constexpr (__is_same(T, ElemBF16))
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                      __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

__device__ const u32x4_t kNothing = {0, 0, 0, 0};

// Columns [0, V) of the layer, a run of blocks of 16 columns to each workgroup.  f
// takes the products of a block: lane l has those of hidden row l % 16 (past the call's
// last row, of that one) with columns v .. v + 3, v = the block's first + 4 (l / 16).
template <class T, class F>
__device__ __forceinline__ void stream_layer(const Lce& a, char* lds, F f)
{
    const uint32_t lane = threadIdx.x % kWave, part = lane / 16, wave = threadIdx.x / kWave;
    const uint32_t V = (uint32_t)a.c.V, D = (uint32_t)a.c.D, turns = (D + kTurn - 1) / kTurn;
    const uint32_t blocks = (V + 15) / 16, per = (blocks + gridDim.x - 1) / gridDim.x;
    const uint32_t first = blockIdx.x * per < blocks ? blockIdx.x * per : blocks;
    const uint32_t own = first + per < blocks ? per : blocks - first;
    // Rounds in which every wave has a block, and then the rest: a block after the other
    // by all waves, or one more round.
    const uint32_t whole = own / kStreamWaves, rest = own % kStreamWaves;
    const bool share = rest * ((turns + kStreamWaves - 1) / kStreamWaves) < turns;
    const uint32_t rounds = whole + (share ? rest : wave < rest);
    const uint32_t turned = (blockIdx.x * kStreamWaves + wave) * 5 % turns;
    // A round: its block, the lane's row of that (past the last column that one again),
    // and this wave's turns along k: the first one, how many, how far apart.
    struct Round {
        uint32_t block, from, count, apart;
        const u32x4_t* row;
    };
    const auto round = [&](uint32_t i) {
        const bool shared = share && i >= whole;
        Round r;
        r.block = first + (shared ? whole * kStreamWaves + i - whole : i * kStreamWaves + wave);
        r.from = shared ? wave : turned;
        r.count = shared ? (turns + kStreamWaves - 1 - wave) / kStreamWaves : turns;
        r.apart = shared ? kStreamWaves : 1;
        const uint32_t v = r.block * 16 + lane % 16;
        r.row = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(a.c.weight) +
                                                 (size_t)(v < V ? v : V - 1) * a.c.ldw * 2) +
                part;
        return r;
    };
    u32x4_t w[2][kAhead];
    const auto request = [&](const u32x4_t* p, uint32_t turn, uint32_t half, u32x4_t (&to)[kAhead]) {
        const uint32_t s = (turn * 2 + half) * kAhead;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            to[i] = *((s + i) * 32 + part * 8 < D ? p + (s + i) * 4 : &kNothing);
    };
    Round now = round(0);
    if (rounds)
        request(now.row, now.from, 0, w[0]);
    // The hidden rows, zeros behind those that count.
    const uint32_t stride = (uint32_t)a.ldh + 16, chunks = (uint32_t)(a.ldh / 16);
    const uint32_t held = (uint32_t)a.c.rows, rows = a.count[0];
#pragma unroll 8
    for (uint32_t i = threadIdx.x; i < held * chunks; i += kStreamThreads)
        *reinterpret_cast<u32x4_t*>(lds + i / chunks * stride + i % chunks * 16) =
            *(i / chunks < rows ? reinterpret_cast<const u32x4_t*>(a.h + i / chunks * a.ldh) + i % chunks
                                : &kNothing);
    f32x4_t* sums = reinterpret_cast<f32x4_t*>(lds + held * stride); // waves x lanes
    __syncthreads();
    const char* mine = lds + (lane % 16 < held ? lane % 16 : held - 1) * stride + part * 16;
    f32x4_t acc;
    const auto multiply = [&](uint32_t turn, uint32_t half, const u32x4_t (&from)[kAhead]) {
        const uint32_t s = (turn * 2 + half) * kAhead;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if ((s + i) * 32 < D)
                acc = mfma16<T>(__builtin_bit_cast(s16x8_t, from[i]),
                                *reinterpret_cast<const s16x8_t*>(mine + (s + i) * 64), acc);
    };
    for (uint32_t i = 0; i < rounds; ++i) {
        const Round next = round(i + 1 < rounds ? i + 1 : i);
        acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t turn = now.from;
        for (uint32_t k = 0; k < now.count; ++k) {
            const bool more = k + 1 < now.count;
            const uint32_t after = turn + now.apart < turns ? turn + now.apart : 0;
            request(now.row, turn, 1, w[1]);
            multiply(turn, 0, w[0]);
            request(more ? now.row : next.row, more ? after : next.from, 0, w[0]);
            multiply(turn, 1, w[1]);
            turn = after;
        }
        if (share && i >= whole) {
            sums[wave * kWave + lane] = acc;
            __syncthreads();
            if (wave == 0) {
#pragma unroll
                for (int x = 1; x < kStreamWaves; ++x)
                    acc += sums[x * kWave + lane];
                f(acc, now.block * 16 + part * 4);
            }
            __syncthreads();
        } else {
            f(acc, now.block * 16 + part * 4);
        }
        now = next;
    }
}

template <class T, bool KEEP>
__global__ __launch_bounds__(kStreamThreads) void lce_stream_stat_kernel(Lce a)
{
    extern __shared__ __align__(16) char buffer[];
    const uint32_t n = threadIdx.x % 16, rows = a.count[0], V = (uint32_t)a.c.V;
    const float c = a.c.scale * kLog2ef;
    const uint32_t target = n < rows ? (uint32_t)a.target[n] : ~0u;
    float m = -INFINITY, s = 0.0f;
    stream_layer<T>(a, buffer, [&](const f32x4_t& z, uint32_t v) {
        if (KEEP && n < rows && v < V)
            *reinterpret_cast<f32x4_t*>(a.z + (size_t)n * a.piece + v) = z;
        float most = m;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            most = fmaxf(most, v + e < V ? z[e] : -INFINITY);
            if (v + e == target)
                a.zt[n] = z[e];
        }
        const float ref = most == -INFINITY ? 0.0f : most;
        s *= __builtin_amdgcn_exp2f((m - ref) * c);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s += v + e < V ? __builtin_amdgcn_exp2f((z[e] - ref) * c) : 0.0f;
        m = most;
    });
    // The workgroup's lanes that have the same row, in order (the sums' LDS).
    constexpr int kParts = kStreamThreads / 16;
    float2* part = reinterpret_cast<float2*>(buffer + a.c.rows * (a.ldh + 16));
    static_assert(kParts * 16 * sizeof(float2) <= kStreamWaves * kWave * sizeof(f32x4_t), "they fit");
    __syncthreads();
    part[threadIdx.x] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x >= 16 || n >= rows)
        return;
    float most = -INFINITY, sum = 0.0f;
    for (int k = 0; k < kParts; ++k)
        most = fmaxf(most, part[k * 16 + n].x);
    const float ref = most == -INFINITY ? 0.0f : most;
    for (int k = 0; k < kParts; ++k)
        sum += part[k * 16 + n].y * __builtin_amdgcn_exp2f((part[k * 16 + n].x - ref) * c);
    a.stat[(size_t)n * a.tiles_v + blockIdx.x] = make_float2(most, sum);
}

// ---- gradients --------------------------------------------------------------

// d from the kept products: eight columns a thread.
template <class T>
__global__ __launch_bounds__(kBlock) void lce_kept_kernel(Lce a, uint32_t blocks)
{
    const uint32_t n = blockIdx.x / blocks, v = (blockIdx.x % blocks * kBlock + threadIdx.x) * 8;
    const uint32_t V = (uint32_t)a.c.V;
    if (n >= a.count[0] || v >= V)
        return;
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(a.z + (size_t)n * a.piece + v);
    // Read once; past V anything.  (1531 rows against 65537 x 1000: 804 us a
    // call so, 831 otherwise.)
    const f32x4_t z[2] = {__builtin_nontemporal_load(p), __builtin_nontemporal_load(p + 1)};
    const float c = a.c.scale * kLog2ef, m = a.m[n], ls = a.ls[n], fa = a.fa[n], fb = a.fb[n];
    const uint32_t target = (uint32_t)a.target[n];
    float d[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        d[e] = fa * __builtin_amdgcn_exp2f(__builtin_fmaf(z[e / 4][e % 4] - m, c, -ls));
        d[e] = v + e == target ? d[e] - fb : d[e];
        d[e] = v + e < V ? d[e] : 0.0f;
    }
    *reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(a.d) + (size_t)n * a.piece + v) = T::pack(d);
}

// d of the piece that starts at column `first`, rows of a.piece elements.
template <class T, class S>
__device__ __forceinline__ void d_tile(const Lce& a, char* buffer, uint32_t first, uint32_t m0,
                                       uint32_t n0)
{
    const uint32_t lds = lds_of(buffer), rows = a.count[0], v0 = first + m0;
    if (n0 >= rows || v0 >= (uint32_t)a.c.V)
        return;
    const Operand W = {static_cast<const char*>(a.c.weight), a.c.ldw * 2, (uint32_t)a.c.V, (uint32_t)a.c.D};
    const Operand H = {a.h, a.ldh, rows, (uint32_t)a.c.D};
    TileAcc<S> acc;
    multiply<T, S, true, true>(acc, W, H, v0, n0, 0, (uint32_t)a.c.D, lds, turn_of<S>(m0 / S::M));

    const float c = a.c.scale * kLog2ef;
    const uint32_t left = (uint32_t)a.c.V - v0;
    float most[S::NS], ls[S::NS], fa[S::NS], fb[S::NS];
    uint32_t at[S::NS];
#pragma unroll
    for (int j = 0; j < S::NS; ++j) {
        const uint32_t n = n0 + acc.n(j);
        const bool in = n < rows;
        most[j] = in ? a.m[n] : 0.0f;
        ls[j] = in ? a.ls[n] : 0.0f;
        fa[j] = in ? a.fa[n] : 0.0f;
        fb[j] = in ? a.fb[n] : 0.0f;
        at[j] = in ? (uint32_t)a.target[n] - v0 : ~0u;
    }
    store_tile<T, false>(acc, lds, S::M, [&](float z, int i, int j, int e) {
        const uint32_t m = acc.m(i, e);
        float d = fa[j] * __builtin_amdgcn_exp2f(__builtin_fmaf(z - most[j], c, -ls[j]));
        d = m == at[j] ? d - fb[j] : d;
        return m < left ? d : 0.0f;
    }, [&](uint32_t n) {
        return reinterpret_cast<uint16_t*>(a.d) + (size_t)(n0 + n) * a.piece + m0;
    });
}

template <class T, class S>
__global__ __launch_bounds__(S::kThreads) void lce_d_kernel(Lce a, uint32_t first, uint32_t tiles)
{
    __shared__ __align__(1024) char buffer[S::kLds];
    with_tile<S>(blockIdx.x, tiles, live_tiles(a, S::N), a.cus, [&](auto shape, uint32_t m, uint32_t n0) {
        d_tile<T, decltype(shape)>(a, buffer, first, m * S::M, n0);
    });
}

// dh [+]= d W over the steps of k of split blockIdx.y.
template <class T, class S>
__global__ __launch_bounds__(S::kThreads) void lce_dh_kernel(Lce a, uint32_t first, uint32_t tiles_m,
                                                             uint32_t tiles_n)
{
    __shared__ __align__(1024) char buffer[S::kLds];
    const uint32_t lds = lds_of(buffer);
    const uint32_t rows = a.count[0], live = live_tiles(a, S::N);
    if (blockIdx.x >= tiles_m * live)
        return;
    const TileAt t = tile_at(in_order(blockIdx.x, tiles_m * live), tiles_m, live);
    const uint32_t m0 = t.m * S::M, n0 = t.n * S::N;
    const uint32_t left = (uint32_t)a.c.V - first, k = left < a.piece ? left : a.piece;
    const uint32_t stages = (k + S::K - 1) / S::K;
    const uint32_t per = (stages + a.splits - 1) / a.splits * S::K;
    const uint32_t begin = blockIdx.y * per < k ? blockIdx.y * per : k;
    const uint32_t end = begin + per < k ? begin + per : k;
    const Operand W = {static_cast<const char*>(a.c.weight) + (size_t)first * a.c.ldw * 2,
                       a.c.ldw * 2, (uint32_t)a.c.D, k};
    const Operand d = {a.d, (size_t)a.piece * 2, rows, k};
    TileAcc<S> acc;
    multiply<T, S, false, true>(acc, W, d, m0, n0, begin, end, lds);
    // In the order of the tile's lanes: 16 bytes a lane, 1 KiB a wave.
    const size_t tile = ((size_t)blockIdx.y * tiles_m + t.m) * tiles_n + t.n;
    f32x4_t* to = reinterpret_cast<f32x4_t*>(a.dh) + tile * (S::M * S::N / 4) +
                  threadIdx.x / kWave * (S::MS * S::NS * 4 * kWave) + threadIdx.x % kWave;
#pragma unroll
    for (int i = 0; i < S::MS; ++i)
#pragma unroll
        for (int j = 0; j < S::NS; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4_t* p = to + ((i * S::NS + j) * 4 + q) * kWave;
                f32x4_t v = {acc.c[i][j][4 * q], acc.c[i][j][4 * q + 1], acc.c[i][j][4 * q + 2],
                             acc.c[i][j][4 * q + 3]};
                if (first)
                    v += *p;
                *p = v;
            }
}

// dh's 32 x 32 blocks, one a workgroup: their splits' sums, in order, rounded once,
// through LDS to the rows of the call.
template <class T, class S>
__global__ __launch_bounds__(kBlock) void lce_dh_finish_kernel(Lce a, uint32_t tiles_m, uint32_t tiles_n,
                                                               uint32_t blocks_m, uint32_t first)
{
    constexpr uint32_t kRow = 32 + 8; // elements of a row in LDS
    __shared__ __align__(16) uint16_t lds[32 * kRow];
    const uint32_t rows = a.count[0];
    const uint32_t n0 = (first + blockIdx.x / blocks_m) * 32, m0 = blockIdx.x % blocks_m * 32;
    if (n0 >= rows)
        return;
    const uint32_t in_m = m0 % S::M, in_n = n0 % S::N;
    const uint32_t wave = in_m / (S::MS * 32) * S::WN + in_n / (S::NS * 32);
    const uint32_t i = in_m / 32 % S::MS, j = in_n / 32 % S::NS;
    const uint32_t q = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const size_t tile = (size_t)(m0 / S::M) * tiles_n + n0 / S::N;
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(a.dh) + tile * (S::M * S::N / 4) +
                       ((wave * S::MS * S::NS + i * S::NS + j) * 4 + q) * kWave + lane;
    const size_t split = (size_t)tiles_m * tiles_n * (S::M * S::N / 4);
    f32x4_t v = *p;
#pragma unroll 8
    for (uint32_t k = 1; k < a.splits; ++k)
        v += p[k * split];
    const uint32_t n = lane % 32;
    const Factor f = n0 + n < rows ? a.fs[n0 + n] : Factor{0.0f, 0};
    uint64_t packed = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x)
        packed |= (uint64_t)(uint16_t)T::narrow(f.times(v[x])) << (16 * x);
    *reinterpret_cast<uint64_t*>(lds + n * kRow + q * 8 + lane / 32 * 4) = packed;
    __syncthreads();
    const uint32_t r = threadIdx.x / 4, c = threadIdx.x % 4 * 8; // D is a multiple of 8
    if (threadIdx.x >= 128 || n0 + r >= rows || m0 + c >= a.c.D)
        return;
    const u32x4_t u = *reinterpret_cast<const u32x4_t*>(lds + r * kRow + c);
    uint16_t* out = static_cast<uint16_t*>(a.c.dhidden) + (size_t)a.row[n0 + r] * a.c.lddh + m0 + c;
    *reinterpret_cast<u32x4u_t*>(out) = u32x4u_t{u.x, u.y, u.z, u.w};
}

// The piece's rows of dW.
template <class T, class S>
__device__ __forceinline__ void dw_tile(const Lce& a, char* buffer, uint32_t first, uint32_t m0,
                                        uint32_t n0)
{
    const uint32_t lds = lds_of(buffer), rows = a.count[0];
    const uint32_t left = (uint32_t)a.c.V - first;
    if (n0 >= left)
        return;
    const Operand H = {a.hs, a.ldh, (uint32_t)(a.ldh / 2), rows};
    const Operand d = {a.d, (size_t)a.piece * 2, a.piece, rows};
    TileAcc<S> acc;
    if constexpr (__is_same(T, ElemF16)) {
        // The groups of rows, from that of the smallest weights on.
        const uint32_t lane = threadIdx.x % kWave, size = lane < kGroups ? a.group[lane] : 0;
        uint32_t end = rows, last = 0;
        acc.clear();
        for (uint64_t left_groups = __ballot(size != 0); left_groups;) {
            const uint32_t g = 63 - __builtin_clzll(left_groups);
            const uint32_t begin = end - __builtin_amdgcn_readlane(size, g);
            if (end != rows)
                acc.scale(ldexpf(1.0f, -(int)(last - g) * kGroupExponents));
            multiply<T, S, false, false, true>(acc, H, d, m0, n0, begin, end, lds);
            end = begin;
            last = g;
            left_groups &= ~(1ull << g);
        }
    } else {
        multiply<T, S, false, false>(acc, H, d, m0, n0, 0, rows, lds);
    }
    const Factor f = factor_of<T>(__uint_as_float(a.count[1]), a.c.scale);
    store_tile<T, true>(acc, lds, (uint32_t)a.c.D - m0,
                        [&](float v, int, int, int) { return f.times(v); },
                        [&](uint32_t n) -> uint16_t* {
                            return n0 + n < left ? static_cast<uint16_t*>(a.c.dweight) +
                                                       (size_t)(first + n0 + n) * a.c.lddw + m0
                                                 : nullptr;
                        });
}

template <class T, class S>
__global__ __launch_bounds__(S::kThreads) void lce_dw_kernel(Lce a, uint32_t first, uint32_t tiles_m,
                                                             uint32_t tiles_n)
{
    __shared__ __align__(1024) char buffer[S::kLds];
    // In halves at most: the tile's rows of d need 128 columns.
    with_tile<S, 2>(blockIdx.x, tiles_m, tiles_n, a.cus, [&](auto shape, uint32_t m, uint32_t n0) {
        dw_tile<T, decltype(shape)>(a, buffer, first, m * S::M, n0);
    });
}

// ---- plan -------------------------------------------------------------------

// Of a piece's d, where that is 2048 columns or more: a piece costs its launches and their
// last rounds of tiles, and past the Infinity Cache d is read from memory.  Bf16, ms with 96,
// 256 and 768 MiB: 4096 x 131072 x 4096 14.6, 14.5, 16.8; 16384 x 32768 x 1024 6.06, 4.57, 4.92;
// 8192 x 131072 x 512 7.01, 5.42, 5.15.
constexpr size_t kPieceBytes = size_t(256) << 20;
constexpr size_t kRowsPad = 256, kColPad = 256; // of rows in the workspace, of a piece
// A launch holds at most 2^32 - 1 work-items, of which a tile takes up to 512.
constexpr uint32_t kTilesPerLaunch = 1u << 22;

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Where the vocabulary is one piece its products (fp32) may be kept from the first pass for
// the gradients: writing and reading them costs less than the layer's rows and the
// products again where the products fit the caches or the rows are wide.  Bf16, us with
// the products kept and computed again:
//    200 x  50001 x  128 (38 MB)     68.5   68.5      1040 x 50001 x  128 (198 MB)   207  183
//    600 x  50001 x  256 (114 MB)    153    160       2000 x 12000 x  256 (96 MB)    142  140
//   1040 x  50001 x  512 (198 MB)    308    329       4000 x 12000 x  512 (192 MB)   297  292
//    136 x  50001 x  512 (26 MB)     106    120       4000 x 12000 x  640 (192 MB)   350  356
//  70000 x   2000 x  512 (560 MB)   2127   2094      70000 x  2000 x  640 (560 MB)  2280 2265
//   1040 x  50001 x 1024 (198 MB)    473    538      70000 x  2000 x 1024 (560 MB)  2431 2518
// So they are kept from this width on, and of narrower rows up to so many bytes for each
// element of a row.  kKeptBytes is for the workspace's sake: one piece takes no more, but for
// more than 65536 rows.
constexpr size_t kKeptBytes = size_t(512) << 20, kKeptWidth = 640, kKeptOfWidth = size_t(384) << 10;

enum class Kind { Few, Mid, Big };

// Tiles by the work: 32 rows by 128 columns where there are few rows, whose product
// only reads the layer, or so little of both that larger tiles leave most compute units
// without one; 256 x 256, the fastest, where every compute unit gets one; 128 x 128 in
// between.  Bf16, both gradients wanted, us with the rule's tile and with its neighbour's:
//   48 x 50001 x 1024        101 (128 x 128)    112 (32 x 128)
//   300 x 4000 x 2048        67.5 (128 x 128)   73.5 (32 x 128)
//   100 x 8000 x 1024        47.7 (32 x 128)    51.5 (128 x 128)
//   600 x 12000 x 1024       104 (128 x 128)    119 (256 x 256)
//   600 x 30000 x 1024       211 (256 x 256)    218 (128 x 128)
struct LcePlan {
    Kind kind, kind_w; // of the products over rows; of the layer's gradient
    uint32_t tiles_v, tiles_n, tiles_d;
    size_t rows, piece, splits, bytes;
    size_t stream_lds;
    bool stream, keep; // the logits by stream_layer; kept
};

template <class F>
auto with_shape(Kind k, F f)
{
    switch (k) {
    case Kind::Few: return f(FewTile());
    case Kind::Mid: return f(MidTile());
    default: return f(BigTile());
    }
}

// Places in the workspace, 256 bytes apart at least; with base null it only adds
// up.
struct Places {
    char* base;
    size_t used = 0;
    template <class P>
    void take(P*& p, size_t bytes)
    {
        p = base ? reinterpret_cast<P*>(base + used) : nullptr;
        used += round_up(bytes, 256);
    }
};

LcePlan plan_of(const LinearCall& c, const DeviceInfo& dev, Lce* a)
{
    LcePlan p;
    const bool grad = c.dhidden || c.dweight;
    Lce dummy;
    Lce& o = a ? *a : dummy;
    p.rows = round_up(c.rows, kRowsPad);
    const size_t big = round_up(c.V, 256) / 256 * (p.rows / 256);
    o.ldh = round_up(c.D, kWidthPad) * 2;
    p.stream_lds = stream_lds(c.rows, o.ldh);
    p.stream = c.rows <= kStreamRowsMax && p.stream_lds <= kStreamLds;
    const size_t mid = round_up(c.V, 128) / 128 * (round_up(c.rows, 128) / 128);
    p.kind = c.rows <= 32 || 4 * mid <= (size_t)dev.cus ? Kind::Few
             : c.rows > 128 && big >= (size_t)dev.cus   ? Kind::Big
                                                        : Kind::Mid;
    size_t tile = 0; // elements
    with_shape(p.kind, [&](auto s) {
        p.tiles_v = (uint32_t)((c.V + s.M - 1) / s.M);
        p.tiles_n = (uint32_t)((c.rows + s.N - 1) / s.N);
        p.tiles_d = (uint32_t)((c.D + s.M - 1) / s.M);
        tile = (size_t)s.M * s.N;
        return 0;
    });
    if (p.stream)
        p.tiles_v = (uint32_t)std::min<size_t>((size_t)dev.cus, (c.V + 15) / 16);
    p.kind_w = c.rows <= 128 || p.kind != Kind::Big ? Kind::Mid : Kind::Big;
    p.piece = std::min(round_up(c.V, kColPad),
                       std::max<size_t>(2048, kPieceBytes / 2 / p.rows / kColPad * kColPad));
    const size_t tiles = (size_t)p.tiles_d * p.tiles_n, stages = p.piece / 64;
    p.splits = std::max<size_t>(1, std::min((size_t)dev.cus / std::max<size_t>(1, tiles), stages / 8));

    Places w = {static_cast<char*>(c.workspace)};
    o.c = c;
    const size_t n = p.rows;
    w.take(o.count, 12);
    w.take(o.group, 4 * kGroups);
    w.take(o.where, 4 * n);
    w.take(o.row, 4 * n);
    w.take(o.target, 4 * n);
    for (float** f : {&o.w, &o.zt, &o.m, &o.ls, &o.fa, &o.fb})
        w.take(*f, 4 * n);
    w.take(o.fs, sizeof(Factor) * n);
    w.take(o.loss_part, 8 * n / kJoinWaves + 8);
    w.take(o.h, o.ldh * n);
    o.hs = nullptr;
    if (c.dweight)
        w.take(o.hs, o.ldh * n);
    o.tiles_v = p.tiles_v;
    w.take(o.stat, sizeof(float2) * p.tiles_v * c.rows);
    o.piece = (uint32_t)p.piece;
    o.splits = (uint32_t)p.splits;
    o.cus = (uint32_t)dev.cus;
    const size_t kept = 4 * p.piece * c.rows;
    p.keep = grad && p.piece >= c.V && kept <= kKeptBytes &&
             (c.D >= kKeptWidth || kept <= c.D * kKeptOfWidth);
    if (p.keep)
        w.take(o.z, kept);
    if (grad)
        w.take(o.d, 2 * p.piece * n);
    if (c.dhidden)
        w.take(o.dh, 4 * p.splits * tiles * tile);
    p.bytes = w.used;
    return p;
}

template <class T>
hipError_t run(const LinearCall& c, const DeviceInfo& dev, hipStream_t s)
{
    Lce a;
    const LcePlan p = plan_of(c, dev, &a);
    const dim3 gather((unsigned)c.rows + kRowPad);
    if (c.rows <= kRowsAlone) {
        hipLaunchKernelGGL((lce_gather_kernel<T, true>), gather, dim3(256), 0, s, a);
    } else {
        if (std::is_same<T, ElemF16>::value && c.dweight)
            hipLaunchKernelGGL(lce_rows_kernel<true>, dim3(1), dim3(1024), 0, s, a);
        else
            hipLaunchKernelGGL(lce_rows_kernel<false>, dim3(1), dim3(1024), 0, s, a);
        hipLaunchKernelGGL((lce_gather_kernel<T, false>), gather, dim3(256), 0, s, a);
    }
    const auto stat = [&](auto keep) {
        constexpr bool KEEP = decltype(keep)::value;
        if (p.stream) {
            hipLaunchKernelGGL((lce_stream_stat_kernel<T, KEEP>), dim3(p.tiles_v),
                               dim3(kStreamThreads), p.stream_lds, s, a);
            return;
        }
        with_shape(p.kind, [&](auto shape) {
            typedef decltype(shape) S;
            const uint32_t most = std::max(8u, kTilesPerLaunch / p.tiles_n);
            for (uint32_t first = 0; first < p.tiles_v; first += most) {
                const uint32_t tiles_m = std::min(most, p.tiles_v - first);
                hipLaunchKernelGGL((lce_stat_kernel<T, S, KEEP>),
                                   dim3(workgroups<S>(tiles_m, p.tiles_n, a.cus)), dim3(S::kThreads),
                                   0, s, a, first, tiles_m);
            }
            return 0;
        });
    };
    if (p.keep)
        stat(std::true_type());
    else
        stat(std::false_type());
    hipLaunchKernelGGL(lce_join_kernel<T>, dim3((unsigned)((c.rows + kJoinWaves - 1) / kJoinWaves)),
                       dim3(kJoinThreads), 0, s, a);
    if (!c.dhidden && !c.dweight)
        return hipGetLastError();
    for (size_t first = 0; first < c.V; first += p.piece) {
        const uint32_t f = (uint32_t)first;
        if (p.keep) {
            const uint32_t blocks = (uint32_t)((c.V + 8 * kBlock - 1) / (8 * kBlock));
            hipLaunchKernelGGL(lce_kept_kernel<T>, dim3((unsigned)c.rows * blocks), dim3(kBlock), 0, s,
                               a, blocks);
        }
        with_shape(p.kind, [&](auto shape) {
            typedef decltype(shape) S;
            const uint32_t tiles_m = (uint32_t)p.piece / S::M;
            if (!p.keep)
                hipLaunchKernelGGL((lce_d_kernel<T, S>),
                                   dim3(workgroups<S>(tiles_m, p.tiles_n, a.cus)), dim3(S::kThreads),
                                   0, s, a, f, tiles_m);
            if (c.dhidden)
                hipLaunchKernelGGL((lce_dh_kernel<T, S>),
                                   dim3(p.tiles_d * p.tiles_n, (unsigned)p.splits),
                                   dim3(S::kThreads), 0, s, a, f, p.tiles_d, p.tiles_n);
            return 0;
        });
        if (c.dweight) {
            const uint32_t cols = (uint32_t)std::min(p.piece, c.V - first);
            const auto dw = [&](auto shape) {
                typedef decltype(shape) S;
                const uint32_t tiles_m = (uint32_t)((c.D + S::M - 1) / S::M);
                const uint32_t tiles_n = (cols + S::N - 1) / S::N;
                hipLaunchKernelGGL((lce_dw_kernel<T, S>),
                                   dim3(workgroups<S>(tiles_m, tiles_n, a.cus)), dim3(S::kThreads), 0,
                                   s, a, f, tiles_m, tiles_n);
            };
            if (p.kind_w == Kind::Mid)
                dw(MidWeight());
            else
                dw(BigTile());
        }
    }
    if (c.dhidden)
        with_shape(p.kind, [&](auto shape) {
            typedef decltype(shape) S;
            const uint32_t blocks_m = (uint32_t)((c.D + 31) / 32);
            const uint32_t blocks_n = (uint32_t)((c.rows + 31) / 32);
            const uint32_t most = std::max(1u, kTilesPerLaunch / blocks_m);
            for (uint32_t first = 0; first < blocks_n; first += most)
                hipLaunchKernelGGL((lce_dh_finish_kernel<T, S>),
                                   dim3(blocks_m * std::min(most, blocks_n - first)), dim3(kBlock), 0,
                                   s, a, p.tiles_d, p.tiles_n, blocks_m, first);
            return 0;
        });
    return hipGetLastError();
}

} // namespace

size_t linear_ce_workspace(const LinearCall& a, const DeviceInfo& dev)
{
    return plan_of(a, dev, nullptr).bytes;
}

hipError_t launch_linear_ce(LogitType t, const LinearCall& a, const DeviceInfo& dev,
                            hipStream_t stream)
{
    return t == LogitType::F16 ? run<ElemF16>(a, dev, stream) : run<ElemBF16>(a, dev, stream);
}

} // namespace red
