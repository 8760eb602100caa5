// The residual's addition, the norm of each token, and 8-bit integers with a scale per token.
#pragma once
#include "rows.cuh"

namespace specs {

struct NormParams {
    Rows x, res, res_out, out;
    const void* weight;
    float* scale;
    long long rows;
    int N, D;
    float eps;
    int norm;      // 0: codes of x as it is
};

// The integer nearest to 127 p / m, even on ties. p and m hold at most 24 significant bits, so the quotient in 64 bits is on
// the side of a half-integer that the exact one is on, and equal to it where that is.
__device__ __forceinline__ int code_exact(float p, float m) {
    return __double2int_rn(127.0 * static_cast<double>(p) / static_cast<double>(m));
}

template <class T, bool CODES>
__global__ void __launch_bounds__(256) norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float s_sum[8];
    __shared__ unsigned s_max[8];
    after_previous();
    const long long t = blockIdx.x;
    const int b = static_cast<int>(t / p.N), n = static_cast<int>(t - static_cast<long long>(b) * p.N);
    const T* const x = row_of<T>(p.x, b, n);
    const T* const res = p.res.p ? row_of<T>(p.res, b, n) : nullptr;
    const T* const w = static_cast<const T*>(p.weight);
    auto value = [&](int i) {
        const T v = x[i];
        return res ? to_float(from_float<T>(to_float(v) + to_float(res[i]))) : to_float(v);
    };
    float sum = 0.f;
    unsigned top = 0u;
    for (int i = threadIdx.x; i < p.D; i += 256) {
        const float r = value(i), q = w ? r * to_float(w[i]) : r;
        sum = fmaf(r, r, sum);
        top = max(top, __float_as_uint(q) & 0x7FFFFFFFu);
    }
    sum = specv::warp_sum(sum);
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum, s_max[threadIdx.x >> 5] = top;
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < 8; ++i) sum += s_sum[i], top = max(top, s_max[i]);
    const float inv = p.norm ? rsqrtf(sum / p.D + p.eps) : 1.f, m = __uint_as_float(top);
    const bool bad = !(m < INFINITY);
    for (int i = threadIdx.x; i < p.D; i += 256) {
        const float r = value(i), q = w ? r * to_float(w[i]) : r;
        if (res) row_of<T>(p.res_out, b, n)[i] = from_float<T>(r);
        if (CODES) row_of<signed char>(p.out, b, n)[i] = static_cast<signed char>(bad || m == 0.f ? 0 : code_exact(q, m));
        else row_of<T>(p.out, b, n)[i] = from_float<T>(q * inv);
    }
    if (CODES && threadIdx.x == 0) p.scale[t] = bad ? NAN : m / 127.f * inv;
}

}  // namespace specs
