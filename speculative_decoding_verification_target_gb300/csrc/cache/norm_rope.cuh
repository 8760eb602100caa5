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
    int N, Hq, Hk, rotary, parts;
    float eps;
};

constexpr int NORM_WARPS = 4;

// A warp takes one token and 1 / parts of its heads, D / 8 lanes to a head with eight channels each: four and the four
// that they are paired with (rotary / 2 further on in the half-split form, the next four otherwise), so that a rotation
// stays within the lane. The token's angles are worked out once per warp: turns = position x frequency in 2^-64 of a
// turn wraps exactly in integer arithmetic, its top 32 bits are the angle to 2^-32 of a turn, so a far position costs no
// precision and no table is read. A lane's channels are the same in every head: y_i = r (x_i P_i + x_mate Q_i), where P
// and Q hold the weights and the cosines and sines, once for the query heads and once for the key heads.
// Bandwidth bounds many tokens: U heads a lane are on their way while U are worked on, the first of them before the angles
// are. 16384 tokens of 32 + 8 heads of 128 in bf16 take 56.4 us, 5.9 TB/s, 89% of the copy rate (70 us
// without the loads ahead, 86 us with a head's eight channels side by side in a lane and shuffles for the rotation); in fp32
// 100.5 us, the copy rate. Few tokens are split into parts; there latency counts: 384 tokens 5.8 us.
// WHOLE: every channel is rotated. Where some are not, their Q is 0, which an infinite mate would turn into a NaN: such rows
// are looked for. (With that in the one kernel for both, the 16384 tokens take 57.0 us where they take 56.4.)
template <class T, int D, bool INTER, bool WHOLE>
__global__ void __launch_bounds__(NORM_WARPS * 32, sizeof(T) == 2 ? 5 : 4) norm_rope_kernel(const __grid_constant__ NormParams p) {
    constexpr int LPH = D / 8, RPW = 32 / LPH;   // lanes per head, heads per warp at a time
    constexpr int U = 4;                         // heads per lane in flight
    constexpr int MATE = INTER ? 1 : 4;
    __shared__ float2 s_cs[NORM_WARPS][D / 2];
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long unit = static_cast<long long>(blockIdx.x) * NORM_WARPS + warp;
    const long long tok = unit / p.parts;
    if (tok >= p.tokens) return;
    const int part = static_cast<int>(unit - tok * p.parts);
    const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok - static_cast<long long>(b) * p.N);
    const int c = lane % LPH, sub = lane / LPH;
    float2* const cs = s_cs[warp];
    const bool rot = WHOLE || 8 * c < p.rotary;
    const int oa = rot && !INTER ? 4 * c : 8 * c, ob = rot && !INTER ? p.rotary / 2 + 4 * c : 8 * c + 4;
    // The part's heads are part RPW + sub + m step, query and key heads in one count; queries first, then keys. A step's
    // heads can straddle the two: a group begins with the step that holds its first head.
    const int H = p.Hq + p.Hk, step = p.parts * RPW, at = part * RPW;
    const int begin_k = at + (p.Hq - RPW + 1 > at ? (p.Hq - RPW + 1 - at + step - 1) / step * step : 0);
    auto row = [&](const Heads& t, int h) { return static_cast<T*>(t.p) + b * t.sb + n * t.sn + h * t.sh; };
    Four<T> na[U], nb[U];      // the next heads, on their way
    auto fetch = [&](int group, int h0) {
        const Heads& in = group ? p.k : p.q;
        const int lo = group ? p.Hq : 0, hi = group ? H : p.Hq;
        const T* src = row(in, h0 + sub - lo);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * step + sub;
            if (h >= lo && h < hi) {
                na[u].load(src + oa);
                nb[u].load(src + ob);
            }
            src += step * in.sh;
        }
    };
    int group = at < p.Hq ? 0 : 1, h0 = group ? begin_k : at;
    if (group && h0 >= H) return;
    fetch(group, h0);          // ahead of the angles
    if (p.rotary) {
        const long long pos = p.positions[tok];
        for (int i = lane; i < p.rotary / 2; i += 32) {
            const unsigned long long turn = static_cast<unsigned long long>(pos) * p.freqs[i];
            const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;   // half turns
            float s, co;
            sincospif(x, &s, &co);
            cs[i] = make_float2(co, s);
        }
        __syncwarp();
    }
    while (true) {
        const int lo = group ? p.Hq : 0, hi = group ? H : p.Hq;
        unsigned long long P[4], Q[4];
        {
            const T* const w = static_cast<const T*>(group ? p.kw : p.qw);
            float wt[8], pc[8], qc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) wt[i] = 1.f;
            if (w) {
                Four<T> e;
                e.load(w + oa);
                e.get(wt);
                e.load(w + ob);
                e.get(wt + 4);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 t = rot ? cs[INTER ? 4 * c + i / 2 : 4 * c + i % 4] : make_float2(1.f, 0.f);
                pc[i] = wt[i] * t.x;
                qc[i] = i & MATE ? wt[i ^ MATE] * t.y : -wt[i ^ MATE] * t.y;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) P[i] = pack2(pc[2 * i], pc[2 * i + 1]), Q[i] = pack2(qc[2 * i], qc[2 * i + 1]);
        }
        const Heads& out = group ? p.ko : p.qo;
        T* dst = row(out, h0 + sub - lo);
        for (; h0 < hi; h0 += U * step) {
            Four<T> ea[U], eb[U];      // a lane without a head computes on what is there: only its own head's lanes see it
#pragma unroll
            for (int u = 0; u < U; ++u) ea[u] = na[u], eb[u] = nb[u];
            if (h0 + U * step < hi) fetch(group, h0 + U * step);
            else if (!group && begin_k < H) fetch(1, begin_k);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h0 + u * step >= hi) break;          // the same for every lane
                float v[8];
                ea[u].get(v);
                eb[u].get(v + 4);
                unsigned long long x[4], m[4], s2 = 0ull;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = pack2(v[2 * i], v[2 * i + 1]);
                    m[i] = pack2(v[2 * i ^ MATE], v[(2 * i + 1) ^ MATE]);
                    s2 = fma2(x[i], x[i], s2);
                }
                const float2 sp = unpack2(s2);
                float s = sp.x + sp.y;
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (!WHOLE && s == INFINITY && !rot) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) m[i] = 0ull;
                }
                const float r = rsqrtf(fmaf(s, 1.f / D, p.eps));
                const unsigned long long r2 = pack2(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = unpack2(mul2(fma2(x[i], P[i], mul2(m[i], Q[i])), r2));
                    v[2 * i] = y.x, v[2 * i + 1] = y.y;
                }
                const int h = h0 + u * step + sub;
                if (h >= lo && h < hi) {
                    ea[u].set(v);
                    ea[u].store(dst + oa);
                    eb[u].set(v + 4);
                    eb[u].store(dst + ob);
                }
                dst += step * out.sh;
            }
        }
        if (group || begin_k >= H) return;
        group = 1;
        h0 = begin_k;
    }
}

}  // namespace specc
