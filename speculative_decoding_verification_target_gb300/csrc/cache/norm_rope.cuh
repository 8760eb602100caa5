// Norm of each query and key head and rotation by position, one pass over the projections.
#pragma once
#include "cache_format.cuh"

namespace specc {

struct NormParams {
    Heads q, k, qo, ko;
    const int* positions;
    const unsigned long long* freqs;
    const void *qw, *kw;
    long long tokens;
    int N, Hq, Hk, rotary, interleaved, parts;
    float eps;
};

constexpr int NORM_WARPS = 4;

// A warp takes one token and 1 / parts of its heads, D / 8 lanes to a head with eight channels each. The token's
// angles are worked out once per warp: turns = position x frequency in 2^-64 of a turn wraps exactly in integer
// arithmetic, its top 32 bits are the angle to 2^-32 of a turn, so a far position costs no precision and no
// table is read. A lane's channels are the same in every head, so it keeps their cosines and sines (and both
// weights) in registers. In the half-split form a pair's two channels sit in lanes rotary / 16 apart.
template <class T, int D>
__global__ void __launch_bounds__(NORM_WARPS * 32) norm_rope_kernel(const __grid_constant__ NormParams p) {
    constexpr int LPH = D / 8, RPW = 32 / LPH;   // lanes per head, heads per warp at a time
    constexpr int U = 2;                         // heads per lane in flight
    __shared__ float2 s_cs[NORM_WARPS][D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long unit = static_cast<long long>(blockIdx.x) * NORM_WARPS + warp;
    const long long tok = unit / p.parts;
    if (tok >= p.tokens) return;
    const int part = static_cast<int>(unit - tok * p.parts);
    const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok - static_cast<long long>(b) * p.N);
    const int c = lane % LPH, sub = lane / LPH;
    const int half = p.rotary >> 1;
    float2* const cs = s_cs[warp];
    if (p.rotary) {
        const long long pos = p.positions[tok];
        for (int i = lane; i < half; i += 32) {
            const unsigned long long turn = static_cast<unsigned long long>(pos) * p.freqs[i];
            const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;   // half turns
            float s, co;
            sincospif(x, &s, &co);
            cs[i] = make_float2(co, s);
        }
        __syncwarp();
    }
    const bool rot = 8 * c < p.rotary;
    float co[8], si[8];
    int mate = lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) co[i] = 1.f, si[i] = 0.f;
    if (rot) {
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 t = cs[4 * c + i];
                co[2 * i] = co[2 * i + 1] = t.x;
                si[2 * i] = -t.y;
                si[2 * i + 1] = t.y;
            }
        } else {
            const bool low = 8 * c < half;
            mate = low ? lane + half / 8 : lane - half / 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 t = cs[(low ? 8 * c : 8 * c - half) + i];
                co[i] = t.x;
                si[i] = low ? -t.y : t.y;
            }
        }
    }
    float qw[8], kw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) qw[i] = kw[i] = 1.f;
    if (p.qw) {
        Eight<T> e;
        e.load(static_cast<const T*>(p.qw) + 8 * c);
        e.get(qw);
    }
    if (p.kw) {
        Eight<T> e;
        e.load(static_cast<const T*>(p.kw) + 8 * c);
        e.get(kw);
    }
    const T* const q = static_cast<const T*>(p.q.p) + b * p.q.sb + n * p.q.sn + 8 * c;
    const T* const k = static_cast<const T*>(p.k.p) + b * p.k.sb + n * p.k.sn + 8 * c;
    T* const qo = static_cast<T*>(p.qo.p) + b * p.qo.sb + n * p.qo.sn + 8 * c;
    T* const ko = static_cast<T*>(p.ko.p) + b * p.ko.sb + n * p.ko.sn + 8 * c;
    const int H = p.Hq + p.Hk, step = p.parts * RPW;
    for (int h0 = part * RPW; h0 < H; h0 += U * step) {
        Eight<T> e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * step + sub;
            if (h < H) e[u].load(h < p.Hq ? q + h * p.q.sh : k + (h - p.Hq) * p.k.sh);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * step + sub;
            float x[8], y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.f;
            if (h < H) e[u].get(x);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            const float r = __frsqrt_rn(fmaf(s, 1.f / D, p.eps));
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (h < p.Hq ? qw[i] : kw[i]);
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], co[i], x[i ^ 1] * si[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], co[i], __shfl_sync(0xffffffffu, x[i], mate) * si[i]);
            }
            if (h < H) {
                e[u].set(y);
                e[u].store(h < p.Hq ? qo + h * p.qo.sh : ko + (h - p.Hq) * p.ko.sh);
            }
        }
    }
}

}  // namespace specc
