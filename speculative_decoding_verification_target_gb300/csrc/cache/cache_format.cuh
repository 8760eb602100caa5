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

// Non-negative fp32 to the nearest scale's bits, ties to even. Above 2^-14 by integer rounding of the float's own
// bits, below it as a multiple of 2^-17 (a carry out of either gives the next scale's bits).
__device__ __forceinline__ int scale_bits(float v) {
    const uint32_t u = __float_as_uint(v);
    const int normal = static_cast<int>((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (112 << 3);
    const int small = __float2int_rn(v * 131072.f);
    return min(v < 6.103515625e-05f ? small : normal, SCALE_TOP);
}
__device__ __forceinline__ float scale_value(int b) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(b << 7)));
}
// Codes + 8 of eight values under scale s, the i-th in bits 4 i; inv the rounded reciprocal of s, or 0 where s is 0.
// Exact arithmetic's codes: x has at most 11 significant bits and s four, so a quotient of at most 7.5 that is no tie lies
// 2^-14 or more from one, and x inv, off by 2^-20, is brought onto the grid of 2^-16 (adding 192, whose last place that is) before
// it is rounded to an integer. Four codes are put together as one fp32 number below 2^16.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float inv) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = __fsub_rn(__fmaf_rn(x[i], inv, 192.f), 192.f);
        const float c = fminf(fmaxf(rintf(q), -7.f), 7.f) + 8.f;
        v[i] = x[i] == x[i] ? c : 8.f;      // a NaN is 0
    }
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w |= static_cast<uint32_t>(fmaf(fmaf(fmaf(v[4 * i + 3], 16.f, v[4 * i + 2]), 16.f, v[4 * i + 1]), 16.f, v[4 * i])) << (16 * i);
    return w;
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
