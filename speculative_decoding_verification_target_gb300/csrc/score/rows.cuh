// Rows of values as the scoring operators take them (include/specscore.h), on the device.
#pragma once
#include "../cache/cache_format.cuh"
#include "specscore.h"

namespace specs {

using specc::after_previous;

// [B, N] rows with element strides
struct Rows {
    void* p;
    long long sb, sn;
};

template <class T>
__device__ __forceinline__ T* row_of(const Rows& t, int b, int n) {
    return static_cast<T*>(t.p) + b * t.sb + n * t.sn;
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_float(float x) {
    if constexpr (std::is_same_v<T, float>) return x;
    else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(x);
    else return __float2bfloat16_rn(x);
}

}  // namespace specs
