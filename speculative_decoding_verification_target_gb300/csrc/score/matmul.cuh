// The product of 8-bit integers with scales for each token and each channel.
#pragma once
#include "rows.cuh"

namespace specs {

struct MatmulParams {
    Rows a, out;
    const signed char* w;
    const float *a_scale, *w_scale, *bias;
    long long w_stride;
    int tokens, N, C, K;
    unsigned* status;
};

// A CTA takes 64 tokens by 64 channels, a thread 4 by 4 of them; 64 of K at a time in shared memory, four to a word.
constexpr int MT = 64, MK = 64, MPAD = MK / 4 + 1;

template <class T>
__global__ void __launch_bounds__(256) matmul_kernel(const __grid_constant__ MatmulParams p) {
    __shared__ int sa[MT * MPAD], sw[MT * MPAD];
    after_previous();
    const int t0 = blockIdx.y * MT, c0 = blockIdx.x * MT, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += MK) {
        for (int i = threadIdx.x; i < MT * MK; i += 256) {
            const int r = i / MK, k = k0 + i % MK;
            signed char va = 0, vw = 0;
            if (k < p.K && t0 + r < p.tokens) va = row_of<signed char>(p.a, (t0 + r) / p.N, (t0 + r) % p.N)[k];
            if (k < p.K && c0 + r < p.C) vw = p.w[static_cast<long long>(c0 + r) * p.w_stride + k];
            reinterpret_cast<signed char*>(sa)[r * MPAD * 4 + i % MK] = va;
            reinterpret_cast<signed char*>(sw)[r * MPAD * 4 + i % MK] = vw;
        }
        __syncthreads();
#pragma unroll 4
        for (int k = 0; k < MK / 4; ++k) {
            int a[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = sa[(ty + 16 * i) * MPAD + k], w[i] = sw[(tx + 16 * i) * MPAD + k];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(a[i], w[j], acc[i][j]);
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + ty + 16 * i, c = c0 + tx + 16 * j;
            if (t >= p.tokens || c >= p.C) continue;
            float y = static_cast<float>(acc[i][j]) * (p.a_scale[t] * p.w_scale[c]);
            if (p.bias) y += p.bias[c];
            row_of<T>(p.out, t / p.N, t % p.N)[c] = from_float<T>(y);
        }
}

}  // namespace specs
