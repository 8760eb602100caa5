// The product of 8-bit integers for up to eight tokens.
#pragma once
#include "rows.cuh"

namespace specs {

struct MatmulParams {
    Rows a, out;
    const signed char* w;
    const float *a_scale, *w_scale, *bias;
    long long w_stride;
    int tokens, N, C, K;
    int k_warps;      // of a CTA's eight: 1, 2, 4 or 8
};

constexpr int MV_WARPS = 8, MV_CH = 4, MV_SMS = 152;      // SMs of the card that the rule for k_warps was measured on

// 16 codes at p, of which `valid` are there; the others are 0. Without alignment only words that hold a valid code are read.
template <bool ALIGNED>
__device__ __forceinline__ void load16(const signed char* p, int valid, int (&x)[4]) {
    if constexpr (ALIGNED) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const int by = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 3);
        const unsigned* const w = reinterpret_cast<const unsigned*>(p - by);
        unsigned v[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) v[i] = 4 * i < by + valid ? __ldg(w + i) : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned y = __funnelshift_r(v[i], v[i + 1], 8 * by);
            const int left = valid - 4 * i;
            x[i] = static_cast<int>(left >= 4 ? y : left <= 0 ? 0u : y & ((1u << (8 * left)) - 1u));
        }
    }
}

// A sum times its scales' product, and with a bias: each step is rounded by itself, in every kernel, so that a token's outputs do not
// depend on how many others are with it.
__device__ __forceinline__ float scaled_sum(int sum, float scale, bool biased, float bias) {
    const float y = __fmul_rn(static_cast<float>(sum), scale);
    return biased ? __fadd_rn(y, bias) : y;
}

// A warp takes four channels and up to TOKENS tokens, its lanes 16 of K each; k_warps of a CTA's warps share their K. Integer
// products four at a time (dp4a, 64 lanes a cycle and SM; the tensor cores' own integer products are no faster here), whole sums in 32
// bits, so their order does not matter. The weights' bytes bound one token (128256 channels of 4096 in 79.8 us, the copy rate), the
// products eight.
template <class T, int TOKENS, bool ALIGNED>
__global__ void __launch_bounds__(MV_WARPS * 32) matvec_kernel(const __grid_constant__ MatmulParams p) {
    __shared__ int s_sum[MV_WARPS][MV_CH * TOKENS];
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kw = warp % p.k_warps, groups = MV_WARPS / p.k_warps;
    const int c0 = (blockIdx.x * groups + warp / p.k_warps) * MV_CH;
    const signed char *w[MV_CH], *a[TOKENS];
#pragma unroll
    for (int i = 0; i < MV_CH; ++i) w[i] = p.w + min(c0 + i, p.C - 1) * p.w_stride;      // past the end the last one once more
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
        const int t = min(j, p.tokens - 1), b = t / p.N;
        a[j] = row_of<signed char>(p.a, b, t - b * p.N);
    }
    int acc[MV_CH][TOKENS] = {};
    constexpr int AHEAD = TOKENS == 1 ? 4 : TOKENS == 8 ? 1 : 2;      // turns whose loads are on their way together
#pragma unroll AHEAD
    for (int k = (kw * 32 + lane) * 16; k < p.K; k += p.k_warps * 512) {
        int x[MV_CH][4];
#pragma unroll
        for (int i = 0; i < MV_CH; ++i) load16<ALIGNED>(w[i] + k, p.K - k, x[i]);
#pragma unroll
        for (int j = 0; j < TOKENS; ++j) {
            int y[4];
            load16<ALIGNED>(a[j] + k, p.K - k, y);
#pragma unroll
            for (int i = 0; i < MV_CH; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][j] = __dp4a(x[i][q], y[q], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < MV_CH; ++i)
#pragma unroll
        for (int j = 0; j < TOKENS; ++j) {
            const int s = __reduce_add_sync(0xffffffffu, acc[i][j]);
            if (lane == 0) s_sum[warp][j * MV_CH + i] = s;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < groups * MV_CH * TOKENS; e += MV_WARPS * 32) {
        const int g = e / (MV_CH * TOKENS), i = e % MV_CH, j = e % (MV_CH * TOKENS) / MV_CH;
        const int c = (blockIdx.x * groups + g) * MV_CH + i, t = j;
        if (c >= p.C || t >= p.tokens) continue;
        int sum = 0;
        for (int q = 0; q < p.k_warps; ++q) sum += s_sum[g * p.k_warps + q][j * MV_CH + i];
        const float bias = p.bias ? p.bias[c] : 0.f;
        row_of<T>(p.out, t / p.N, t % p.N)[c] = from_float<T>(scaled_sum(sum, p.a_scale[t] * p.w_scale[c], p.bias != nullptr, bias));
    }
}

}  // namespace specs
