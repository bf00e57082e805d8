// mfma_tile.hpp -- products of 16-bit matrices by the matrix cores of gfx950:
// a workgroup's tile C[n][m] = sum_k A(m, k) B(n, k), in fp32.
//
// Each operand lies in memory either with its contraction index contiguous
// ("row" form, A[m][k]) or with the other one ("column" form, A[k][m]).  Tiles
// of K steps of k go from memory to LDS without passing registers
// (buffer_load ... lds, 16 bytes a lane, 1 KiB a wave), into a ring of STAGES
// buffers, and from there to the operand registers of v_mfma_f32_32x32x16:
// by ds_read_b128 from row form, by ds_read_b64_tr_b16, which transposes 4 x 16
// elements among 16 lanes, from column form.
//
// The loads write LDS in lane order, so 16-byte chunks are permuted on the
// memory side instead, to where 16 lanes that read at once find 64 banks:
//   row form    (2 K bytes a row)        chunk c of row r at c ^ row_swizzle(r)
//   column form (2 M bytes a step of k)  chunk c of step k at c ^ 4 (k & 3)
//
// Elements outside an operand are zeros: their lanes load from past the end of
// the buffer descriptor, which gives zeros, so nothing outside is read.
// What bounds it: 256 x 256 tiles of 64 steps keep the matrix cores busy in 66 % of the
// cycles, at a clock that the power limit sets (3584 rows against 131072 x 4096, with the
// rows' sums of exponentials: 3.06 ms, 1.26 PFLOP/s; the library's product of 4096 rows
// alone, 1.44).  8 waves of 128 x 64 with two buffers: 13.0 ms for that loss with its
// gradients; 4 waves of 128 x 128 14.7; steps of 32 in 3 to 5 buffers 13.4; tiles of 256 x 128
// 16.5, 128 x 128 15.9.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "elements.hpp"

namespace red {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// Row form: the rows of 256 bytes share the permutation, the next rows have others.
template <int K>
__device__ __forceinline__ constexpr uint32_t row_swizzle(uint32_t r)
{
    constexpr uint32_t kRows = K < 128 ? 128 / K : 1, kMask = K / 8 < 16 ? K / 8 - 1 : 15;
    return r / kRows & kMask;
}

template <class T>
__device__ __forceinline__ f32x16_t mfma(const s16x8_t& a, const s16x8_t& b, const f32x16_t& c)
{
    if constexpr (__is_same(T, ElemBF16))
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                      __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// A matrix in memory.  `count` rows (m or n) of `k` elements each; ld: bytes
// from one row (row form) or one step of k (column form) to the next.
struct Operand {
    const char* p;
    size_t ld;
    uint32_t count, k;
};

constexpr uint32_t kOutside = 0x80000000u; // past every descriptor's end

// 16 bytes a lane from memory to LDS (lds: the wave's first byte).  The compiler
// does not count these loads: wait_loads() does, before the barrier that makes
// them known to the other waves.  (With the builtin it waited for all of them
// before every transposing read.)
__device__ __forceinline__ void load_to_lds(const u32x4_t& rsrc, uint32_t offset, uint32_t lds)
{
    // Four idle steps: a descriptor that the vector unit wrote is read five steps
    // later at the earliest, and m0 one after it was written.
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(offset), "s"(rsrc)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
constexpr int kLdsDone = 0xc07f; // lgkmcnt(0) alone
__device__ __forceinline__ void barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(kLdsDone);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// One operand's tile of R rows by K.
template <int R, int K, bool ROW, int WAVES>
struct TileOperand {
    static constexpr int kBytes = R * K * 2;
    static constexpr int kLoads = kBytes / 1024 / WAVES;
    static_assert(kLoads >= 1 && kLoads * WAVES * 1024 == kBytes, "whole loads for every wave");
    static constexpr int kChunks = ROW ? K / 8 : R / 8; // of a row, or of a step of k
    static_assert(ROW || kChunks % 16 == 0, "the permutation stays in the step of k");

    uint32_t offset[kLoads], k_of[kLoads]; // of this lane's chunk: bytes from `at`, step of k
    uint64_t at;
    uint64_t advance;
    uint32_t k;

    // first: the tile's first row; begin, end: its steps of k (in row form begin is
    // a multiple of 8).
    __device__ __forceinline__ TileOperand(const Operand& o, uint32_t first, uint32_t begin,
                                           uint32_t end)
    {
        const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
        k = end - begin;
        if constexpr (ROW) {
            at = (uint64_t)o.p + (uint64_t)first * o.ld + (uint64_t)begin * 2;
            advance = K * 2;
        } else {
            at = (uint64_t)o.p + (uint64_t)begin * o.ld + (uint64_t)first * 2;
            advance = (uint64_t)K * o.ld;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t s = (i * WAVES + wave) * kWave + lane;
            if constexpr (ROW) {
                const uint32_t r = s / kChunks, c = (s % kChunks) ^ row_swizzle<K>(r);
                k_of[i] = c * 8;
                offset[i] = first + r < o.count ? r * (uint32_t)o.ld + c * 16 : kOutside;
            } else {
                const uint32_t kk = s / kChunks;
                const uint32_t c = (s % kChunks) ^ ((kk & 3) << 2);
                k_of[i] = kk;
                offset[i] = first + c * 8 < o.count ? kk * (uint32_t)o.ld + c * 16 : kOutside;
            }
        }
    }

    // The descriptor of stage number `stage`.
    __device__ __forceinline__ u32x4_t stage(uint32_t stage) const
    {
        const uint64_t p = at + advance * stage;
        u32x4_t rsrc;
        rsrc.x = __builtin_amdgcn_readfirstlane((uint32_t)p);
        rsrc.y = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32) & 0xffffu);
        rsrc.z = 0x7fffffffu;
        rsrc.w = 0x00020000u;
        return rsrc;
    }
    // Requests load i of stage number `stage` (rsrc) into LDS at `lds`; zeros where
    // not `wanted`.
    __device__ __forceinline__ void request(const u32x4_t& rsrc, int i, uint32_t stage, bool wanted,
                                            uint32_t lds) const
    {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        load_to_lds(rsrc, stage * K + k_of[i] < (wanted ? k : 0) ? offset[i] : kOutside,
                    lds + (i * WAVES + wave) * 1024);
    }

    // The operand registers of 32 rows from `row` (a multiple of 32) on, steps
    // 16 kk to 16 kk + 15 of the stage at `lds`.
    static __device__ __forceinline__ s16x8_t read(uint32_t lds, uint32_t row, int kk)
    {
        const uint32_t lane = threadIdx.x % kWave, half = lane / 32;
        if constexpr (ROW) {
            const uint32_t r = lane % 32;
            const uint32_t a =
                lds + (row + r) * (K * 2) + ((kk * 2 + half) ^ row_swizzle<K>(r)) * 16;
            return *(__attribute__((address_space(3))) const s16x8_t*)(uintptr_t)a;
        } else {
            typedef __attribute__((address_space(3))) s16x4_t* ptr;
            const uint32_t i = lane % 16, c = row / 8 + (lane / 16 % 2) * 2 + (i & 3) / 2;
            const uint32_t a = lds + (kk * 16 + half * 8 + i / 4) * (R * 2) +
                               (c ^ (i / 4 << 2)) * 16 + (i & 1) * 8;
            const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(uintptr_t)a);
            const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(uintptr_t)(a + 4 * (R * 2)));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

// The shape of a workgroup's tile: M x N elements by WM x WN waves, STAGES buffers
// of K steps in LDS.
template <int M_, int N_, int WM_, int WN_, int K_, int STAGES_>
struct TileShape {
    static constexpr int M = M_, N = N_, WM = WM_, WN = WN_, K = K_, STAGES = STAGES_;
    static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
    static constexpr int MS = M / WM / 32, NS = N / WN / 32; // 32 x 32 blocks of a wave
    static constexpr int kStage = (M + N) * K * 2;
    // The finished tile passes through LDS too: rows of M 16-bit elements.
    static constexpr int kOutRow = M * 2 + 16;
    static constexpr int kLds = kStage * STAGES > kOutRow * N ? kStage * STAGES : kOutRow * N;
    static_assert(kLds <= 160 * 1024, "LDS of a compute unit");
};

// c[i][j]: block i of the wave's rows m, block j of its rows n.  Lane l holds
// n = 32 j + l % 32 and, in element e, m = 32 i + 8 (e / 4) + 4 (l / 32) + e % 4.
template <class S>
struct TileAcc {
    f32x16_t c[S::MS][S::NS];
    static __device__ __forceinline__ uint32_t wave_m() { return threadIdx.x / kWave / S::WN * (S::MS * 32); }
    static __device__ __forceinline__ uint32_t wave_n() { return threadIdx.x / kWave % S::WN * (S::NS * 32); }
    static __device__ __forceinline__ uint32_t m(int i, int e)
    {
        return wave_m() + i * 32 + (e / 4) * 8 + threadIdx.x % kWave / 32 * 4 + e % 4;
    }
    static __device__ __forceinline__ uint32_t n(int j) { return wave_n() + j * 32 + threadIdx.x % 32; }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < S::MS; ++i)
#pragma unroll
            for (int j = 0; j < S::NS; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    c[i][j][e] = 0.0f;
    }
    __device__ __forceinline__ void scale(float f)
    {
#pragma unroll
        for (int i = 0; i < S::MS; ++i)
#pragma unroll
            for (int j = 0; j < S::NS; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    c[i][j][e] *= f;
    }
};

// The tile at (m0, n0) over steps [begin, end) of k, in the order of the stages from
// number `turn` on and round.  (Workgroups that read rows of the same length from
// memory in step ask the same few channels at a time; different turns spread them.)
// MORE: added to what acc holds.
template <class T, class S, bool AROW, bool BROW, bool MORE = false>
__device__ __forceinline__ void multiply(TileAcc<S>& acc, const Operand& a, const Operand& b,
                                         uint32_t m0, uint32_t n0, uint32_t begin, uint32_t end,
                                         uint32_t lds, uint32_t turn = 0)
{
    typedef TileOperand<S::M, S::K, AROW, S::kWaves> A;
    typedef TileOperand<S::N, S::K, BROW, S::kWaves> B;
    const A ta(a, m0, begin, end);
    const B tb(b, n0, begin, end);
    const uint32_t stages = (end - begin + S::K - 1) / S::K;
    if constexpr (!MORE)
        acc.clear();
    const uint32_t wm = __builtin_amdgcn_readfirstlane(TileAcc<S>::wave_m());
    const uint32_t wn = __builtin_amdgcn_readfirstlane(TileAcc<S>::wave_n());
    constexpr int kSteps = S::K / 16, kLoads = A::kLoads + B::kLoads;
    // Turn number s works on stage (s + turn) mod stages.
    const uint32_t from = turn % (stages ? stages : 1);
    const auto stage_of = [&](uint32_t s) { return s + from < stages ? s + from : s + from - stages; };
    // Load i of turn s, A's first; past the last turn it brings zeros.
    const auto request = [&](const u32x4_t& ra, const u32x4_t& rb, int i, uint32_t s, uint32_t buffer) {
        const uint32_t at = lds + buffer * S::kStage, stage = stage_of(s);
        if (i < A::kLoads)
            ta.request(ra, i, stage, s < stages, at);
        else
            tb.request(rb, i - A::kLoads, stage, s < stages, at + A::kBytes);
    };
    // Two sets of operand registers: while one is multiplied the other is read.
    s16x8_t fa[2][S::MS], fb[2][S::NS];
    const auto read = [&](uint32_t buffer, int kk) {
        const uint32_t at = lds + buffer * S::kStage;
#pragma unroll
        for (int j = 0; j < S::NS; ++j)
            fb[kk & 1][j] = B::read(at + A::kBytes, wn + j * 32, kk);
#pragma unroll
        for (int i = 0; i < S::MS; ++i)
            fa[kk & 1][i] = A::read(at, wm + i * 32, kk);
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int s = 0; s < S::STAGES; ++s) {
        const u32x4_t ra = ta.stage(stage_of(s)), rb = tb.stage(stage_of(s));
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            request(ra, rb, i, s, s);
    }
    wait_loads<(S::STAGES - 1) * kLoads>();
    barrier();
    read(0, 0);
    __builtin_amdgcn_s_waitcnt(kLdsDone); // or the loop's first wait is for all its reads
    uint32_t cur = 0; // this stage's buffer
    for (uint32_t s = 0; s < stages; ++s) {
        const uint32_t next = cur + 1 == S::STAGES ? 0 : cur + 1;
#pragma unroll
        for (int kk = 0; kk < kSteps - 1; ++kk) {
            read(cur, kk + 1);
#pragma unroll
            for (int i = 0; i < S::MS; ++i)
#pragma unroll
                for (int j = 0; j < S::NS; ++j)
                    acc.c[i][j] = mfma<T>(fa[kk & 1][i], fb[kk & 1][j], acc.c[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        // This wave has read all of the stage, and its loads of the next have landed;
        // behind the barrier that goes for every wave, so the buffer can take another
        // stage while this one's last step is multiplied, a load behind each product.
        wait_loads<(S::STAGES - 2) * kLoads>();
        barrier();
        read(next, 0);
        const u32x4_t ra = ta.stage(stage_of(s + S::STAGES));
        const u32x4_t rb = tb.stage(stage_of(s + S::STAGES));
        constexpr int last = (kSteps - 1) & 1;
        int load = 0;
#pragma unroll
        for (int i = 0; i < S::MS; ++i)
#pragma unroll
            for (int j = 0; j < S::NS; ++j) {
                acc.c[i][j] = mfma<T>(fa[last][i], fb[last][j], acc.c[i][j]);
                __builtin_amdgcn_sched_barrier(0);
                if (load < kLoads)
                    request(ra, rb, load++, s + S::STAGES, cur);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i >= S::MS * S::NS)
                request(ra, rb, i, s + S::STAGES, cur);
        __builtin_amdgcn_sched_barrier(0);
        cur = next;
    }
    // The last requests brought zeros to buffers that are not read; they have
    // landed, and every wave is done reading, before LDS is used otherwise.
    wait_loads<0>();
    barrier();
}

// The tile as 16-bit elements f(value, i, j, e), to rows n of memory:
// row(n) gives a row's first element for column m0, or null.  cols: valid columns.
// PASS: nobody reads them soon, they pass the caches by.
template <class T, bool PASS, class S, class F, class Rows>
__device__ __forceinline__ void store_tile(const TileAcc<S>& acc, uint32_t lds, uint32_t cols, F f,
                                           Rows row)
{
    typedef __attribute__((address_space(3))) uint64_t* ptr8;
    typedef __attribute__((address_space(3))) const u32x4_t* ptr16;
#pragma unroll
    for (int i = 0; i < S::MS; ++i)
#pragma unroll
        for (int j = 0; j < S::NS; ++j)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                uint64_t q = 0;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    q |= (uint64_t)(uint16_t)T::narrow(f(acc.c[i][j][e + x], i, j, e + x)) << (16 * x);
                *(ptr8)(uintptr_t)(lds + acc.n(j) * S::kOutRow + acc.m(i, e) * 2) = q;
            }
    barrier();
    constexpr int kPerRow = S::M / 8; // threads of a row
#pragma unroll
    for (int p = 0; p < S::N * kPerRow / S::kThreads; ++p) {
        const uint32_t x = p * S::kThreads + threadIdx.x, n = x / kPerRow, c = x % kPerRow;
        uint16_t* out = row(n);
        if (!out || c * 8 >= cols)
            continue;
        const u32x4_t v = *(ptr16)(uintptr_t)(lds + n * S::kOutRow + c * 16);
        if (c * 8 + 8 <= cols) {
            if constexpr (PASS)
                __builtin_nontemporal_store(u32x4u_t{v.x, v.y, v.z, v.w},
                                            reinterpret_cast<u32x4u_t*>(out + c * 8));
            else
                *reinterpret_cast<u32x4u_t*>(out + c * 8) = u32x4u_t{v.x, v.y, v.z, v.w};
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c * 8 + k < cols)
                    out[c * 8 + k] = (uint16_t)(v[k / 2] >> (16 * (k % 2)));
        }
    }
}

} // namespace red
