// The 4-bit cache's format (include/speccache.h) on the device, and the element types of the activations.
#pragma once
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../device_common.cuh"
#include "speccache.h"

namespace specc {

constexpr int PAGE = SPEC_CACHE_PAGE;
constexpr int GROUP = SPEC_CACHE_GROUP;
constexpr int SCALE_TOP = 198;            // bits of the largest scale, 896: 72 x 896 is still a finite half

// Every kernel here is launched so that its CTAs may take their places before the kernel in front of it has ended, and begins
// with this: it waits for that end (so for all that came before, since that kernel waited likewise), and lets the next one's
// CTAs in. Nothing in global memory is read or written before it.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// Byte offsets of a block's four parts for head size D.
template <int D>
struct Block {
    static constexpr int NG = D / GROUP;
    static constexpr int KS = 32 * D, V = 34 * D, VS = 66 * D, BYTES = 68 * D;
    __host__ __device__ static constexpr int key(int g, int t) { return (g * PAGE + t) * 16; }
    __host__ __device__ static constexpr int value(int t, int r) { return V + (t / 16) * (8 * D) + r * 16 + t % 16; }
};

// [B, N, heads, D] with element strides
struct Heads {
    void* p;
    long long sb, sn, sh;
};

__device__ __forceinline__ float scale_value(int b) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(b << 7)));
}

// Bits of the scale nearest (even on ties) to a seventh of `top`, the group's largest magnitude, a bf16 or fp16 value. The
// seventh need not be the correctly rounded quotient: top has at most 11 significant bits, so a quotient that is no tie
// between two scales is 2^-15 of itself or more away from one, and the product, off by 2^-23, is first rounded to 16 bits (by
// adding and taking away 2^8 of itself). Above 2^-14 by integer rounding of the float's own bits, below as a multiple of
// 2^-17 (a carry out of either gives the next scale's bits).
__device__ __forceinline__ int scale_bits(float top) {
    const float t = fminf(top, 8192.f) * 0.14285714924335479736328125f, far = t * 257.f;
    const float v = __fsub_rn(far, __fsub_rn(far, t));
    const uint32_t u = __float_as_uint(v);
    const int normal = static_cast<int>((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (112 << 3);
    const int small = __float2int_rn(v * 131072.f);
    return min(v < 6.103515625e-05f ? small : normal, SCALE_TOP);
}

// Codes + 8 of eight values (no NaN) under scale s, the i-th in bits 4 i. Exact arithmetic's codes: x has at most 11
// significant bits and s four, so a quotient of at most 7.5 that is no tie lies 2^-14 or more from one; x times the approximate
// reciprocal is off by 2^-19 and is brought onto the grid of 2^-16 (by adding 192, whose last place that is). Adding
// 1.5 2^23 then rounds to an integer, ties to even, which stands in the last bits of the sum: they are put together as they are,
// and what the sums' upper bits add up to is taken away at once.
// LIMIT: quotients may pass 7.5 (only where the scale is not the nearest 4-bit number to top / 7: in the subnormal range or at
// its top; elsewhere top / s is at most 7 (1 + 1 / 16)).
template <bool LIMIT>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float s) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    inv = s > 0.f ? inv : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float q = __fmaf_rn(x[i], inv, 192.f);
        if (LIMIT) q = fminf(fmaxf(q, 185.f), 199.f);
        w += __float_as_uint(__fadd_rn(q, 12582912.f - 184.f)) << (4 * i);
    }
    return w - 0x3F400000u;      // the sum of 0x4B400000 << 4 i, modulo 2^32
}

// Two fp32 values in one 64-bit register pair: one instruction for both.
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Eight neighbouring channels: 16 bytes of bf16 or fp16.
template <class T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 r;
    __device__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ void set(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
};
template <>
struct Eight<__half> {
    uint4 r;
    __device__ void load(const __half* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    __device__ void set(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ void store(__half* p) const { *reinterpret_cast<uint4*>(p) = r; }
};
// Four neighbouring channels: 8 bytes of bf16 or fp16, 16 of fp32.
template <class T>
struct Four {
    uint2 r;
    __device__ void load(const T* p) { r = *reinterpret_cast<const uint2*>(p); }
    __device__ void get(float* x) const {
        const uint32_t w[2] = {r.x, r.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (std::is_same_v<T, __half>) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                x[2 * i] = f.x, x[2 * i + 1] = f.y;
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
    __device__ void set(const float* x) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (std::is_same_v<T, __half>) {
                const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        r = make_uint2(w[0], w[1]);
    }
    __device__ void store(T* p) const { *reinterpret_cast<uint2*>(p) = r; }
};
template <>
struct Four<float> {
    float4 r;
    __device__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
    __device__ void get(float* x) const { x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w; }
    __device__ void set(const float* x) { r = make_float4(x[0], x[1], x[2], x[3]); }
    __device__ void store(float* p) const { *reinterpret_cast<float4*>(p) = r; }
};

}  // namespace specc
