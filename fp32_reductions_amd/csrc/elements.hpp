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

} // namespace red
