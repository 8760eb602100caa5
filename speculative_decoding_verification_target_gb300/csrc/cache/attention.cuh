// Attention of the newest tokens over the 4-bit cache.
#pragma once
#include "cache_format.cuh"

namespace specc {

struct AttnParams {
    Heads q, out;
    const unsigned char* pool;
    const int* table;
    const int *kv_len, *q_len;
    float* lse;
    unsigned* status;
    int pages, max_pages, B, N, Hq, Hk, window, sinks;
    float scale;             // times log2 e
};

// One warp to a query row: a pass over the visible tokens with the running maximum and sum of the softmax.
template <class T, int D>
__global__ void __launch_bounds__(128) attention_kernel(const __grid_constant__ AttnParams p) {
    using BL = Block<D>;
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.B) * p.N * p.Hq) return;
    const int hq = static_cast<int>(row % p.Hq), i = static_cast<int>(row / p.Hq % p.N), b = static_cast<int>(row / p.Hq / p.N);
    const int h = hq / (p.Hq / p.Hk);
    int ql = p.q_len ? p.q_len[b] : p.N;
    if (ql < 0 || ql > p.N) atomicOr(p.status, SPEC_STATUS_BAD_LENGTH), ql = min(max(ql, 0), p.N);
    int len = p.kv_len[b];
    const long long room = static_cast<long long>(p.max_pages) * PAGE;
    if (len < 0 || len > room) atomicOr(p.status, SPEC_STATUS_BAD_LENGTH), len = static_cast<int>(min(static_cast<long long>(max(len, 0)), room));
    const int pos = i < ql ? len - ql + i : -1;
    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = static_cast<float>(static_cast<const T*>(p.q.p)[b * p.q.sb + i * p.q.sn + hq * p.q.sh + e * 32 + lane]);
        o[e] = 0.f;
    }
    float m = -1e30f, l = 0.f;
    for (int t = 0; t <= pos; ++t) {
        if (p.window > 0 && t >= p.sinks && t <= pos - p.window) continue;
        const int page = p.table[static_cast<size_t>(b) * p.max_pages + t / PAGE];
        if (page < 0 || page >= p.pages) {
            if (lane == 0) atomicOr(p.status, SPEC_STATUS_BAD_PAGE);
            continue;
        }
        const unsigned char* const blk = p.pool + (static_cast<size_t>(page) * p.Hk + h) * BL::BYTES;
        float s = 0.f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = e * 32 + lane, kb = blk[BL::key(e, t % PAGE) + lane / 2], vb = blk[BL::value(t % PAGE, d % (D / 2))];
            s += q[e] * (static_cast<float>(((lane & 1) ? kb >> 4 : kb & 15) - 8) * scale_value(blk[BL::KS + t % PAGE * BL::NG + e]));
            v[e] = static_cast<float>((d < D / 2 ? vb & 15 : vb >> 4) - 8) * scale_value(blk[BL::VS + t % PAGE * BL::NG + e]);
        }
        s = specv::warp_sum(s) * p.scale;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * v[e];
        m = mn;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        static_cast<T*>(p.out.p)[b * p.out.sb + i * p.out.sn + hq * p.out.sh + e * 32 + lane] = static_cast<T>(l > 0.f ? o[e] / l : 0.f);
    if (p.lse && lane == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : __uint_as_float(0xFF800000u);
}

}  // namespace specc
