// elements.hpp -- the element types of matrices whose rows are reduced: 16-byte
// vectors of fp32, fp16 or bf16, widened exactly to fp32 and rounded once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"

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

// Rows need not be aligned to more than their elements: gfx950 loads and
// stores unaligned 16-byte vectors in global memory.
typedef unsigned u32x4u_t __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ void store_vec(void* p, const u32x4_t& v)
{
    u32x4u_t u;
    u.x = v.x; u.y = v.y; u.z = v.z; u.w = v.w;
    __builtin_nontemporal_store(u, reinterpret_cast<u32x4u_t*>(p));
}

// The last `rest` elements of a row (fewer than a vector), packed from its first
// byte on, zeros behind them: p is the first of them.  Where the row is at least a
// vector long (`whole`), one load that ends with the row, shifted; elements one by
// one otherwise.
template <class T>
__device__ __forceinline__ u32x4_t load_rest(const typename T::S* p, uint32_t rest, bool whole)
{
    typedef unsigned __int128 u128;
    if (whole) {
        const u32x4u_t u = *reinterpret_cast<const u32x4u_t*>(p + rest - T::W);
        const u128 v = __builtin_bit_cast(u128, u32x4_t{u.x, u.y, u.z, u.w});
        return __builtin_bit_cast(u32x4_t, v >> (8 * sizeof(typename T::S) * (T::W - rest)));
    }
    float f[T::W];
#pragma unroll
    for (int i = 0; i < T::W; ++i)
        f[i] = i < (int)rest ? T::widen(p[i]) : 0.0f;
    return T::pack(f);
}

// Stores the first `rest` elements of v at p, in pieces of 8, 4 and 2 bytes.
template <class T>
__device__ __forceinline__ void store_rest(typename T::S* p, const u32x4_t& v, uint32_t rest)
{
    typedef unsigned u32x2u_t __attribute__((ext_vector_type(2), aligned(2)));
    typedef unsigned u32u_t __attribute__((aligned(2)));
    const uint32_t bytes = rest * (uint32_t)sizeof(typename T::S);
    char* q = reinterpret_cast<char*>(p);
    if (bytes & 8)
        *reinterpret_cast<u32x2u_t*>(q) = u32x2u_t{v.x, v.y};
    if (bytes & 4)
        *reinterpret_cast<u32u_t*>(q + (bytes & 8)) = bytes & 8 ? v.z : v.x;
    if (bytes & 2)
        *reinterpret_cast<uint16_t*>(q + (bytes & 12)) =
            (uint16_t)((bytes & 8) ? ((bytes & 4) ? v.w : v.z) : ((bytes & 4) ? v.y : v.x));
}

} // namespace red
