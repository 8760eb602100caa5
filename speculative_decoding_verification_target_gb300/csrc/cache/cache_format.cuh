// The 4-bit cache's format (include/speccache.h) on the device, and the element types of the activations.
#pragma once
#include <cstdint>
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
// Code + 8 of x under scale s. The quotient is the correctly rounded one: x has at most 11 significant bits and
// s four, so x / s is a tie exactly where the true quotient is one, and the code is that of exact arithmetic.
__device__ __forceinline__ uint32_t code_of(float x, float s) {
    const float c = s > 0.f && x == x ? rintf(__fdiv_rn(x, s)) : 0.f;   // a NaN is 0
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(c, -7.f), 7.f)) + 8);
}

// Eight neighbouring channels: 16 bytes of bf16 or fp16, 32 of fp32.
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
template <>
struct Eight<float> {
    float4 a, b;
    __device__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ void set(const float (&x)[8]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
    __device__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
};

}  // namespace specc
