// New keys and values quantised into their pages, and cached ones read back.
#pragma once
#include "cache_format.cuh"

namespace specc {

struct TokensParams {
    unsigned char* pool;
    const int* table;
    const int *start, *counts;
    Heads k, v;
    int pages, max_pages, B, N, Hk;
    unsigned* status;
};

constexpr int TOK_THREADS = 256;

// The part of a sequence's new tokens that one CTA (blockIdx: head, page among the new ones, sequence) works on:
// tokens [t0, t1) of page `page`, the first of them being input i0. False where there is none.
struct Span {
    int page, t0, t1, i0;
};
__device__ __forceinline__ bool span_of(const TokensParams& p, int b, int y, bool report, Span& s) {
    const int start = p.start[b];
    int cnt = p.counts ? p.counts[b] : p.N;
    if (cnt < 0 || cnt > p.N) {
        if (report) atomicOr(p.status, SPEC_STATUS_BAD_LENGTH);
        cnt = min(max(cnt, 0), p.N);
    }
    if (cnt == 0) return false;
    // positions below 0 or past the table hold no page
    const long long end = static_cast<long long>(start) + cnt, room = static_cast<long long>(p.max_pages) * PAGE;
    const long long lo = max(start, 0);
    const long long hi = min(end, room);
    if ((start < 0 || end > room) && report) atomicOr(p.status, SPEC_STATUS_BAD_LENGTH);
    const long long j = lo / PAGE + y;
    if (j * PAGE >= hi) return false;
    s.t0 = static_cast<int>(max(lo - j * PAGE, 0LL));
    s.t1 = static_cast<int>(min(hi - j * PAGE, static_cast<long long>(PAGE)));
    s.i0 = static_cast<int>(j * PAGE + s.t0 - start);
    s.page = p.table[static_cast<size_t>(b) * p.max_pages + j];
    if (s.page < 0 || s.page >= p.pages) {
        if (report) atomicOr(p.status, SPEC_STATUS_BAD_PAGE);
        s.page = -1;
    }
    return true;
}

// One CTA quantises the tokens of one page and head; no two CTAs write a byte of the same token, so pages that start or end
// inside the call's range need no read. D / 8 lanes take a token, four of them a group. Keys go to the page as they come:
// two tokens of a warp fill a sector of each group. A value's codes lie with those of 15 other tokens, so they pass through
// shared memory: there as words of eight channels by token, from there a thread gathers the 16 tokens of a byte row, two
// channels, and writes 16 bytes (or, in a run that the range does not fill, the bytes that are its own).
template <class T, int D>
__global__ void __launch_bounds__(TOK_THREADS) append_kernel(const __grid_constant__ TokensParams p) {
    using B = Block<D>;
    constexpr int LPT = D / 8, PER = TOK_THREADS / LPT;      // lanes of a token, tokens of a pass
    constexpr int U = 4;                                     // passes whose loads are in flight together
    __shared__ uint32_t s_codes[PAGE][LPT];
    const int h = blockIdx.x, b = blockIdx.z, tid = threadIdx.x;
    Span sp;
    if (!span_of(p, b, blockIdx.y, h == 0 && tid == 0, sp) || sp.page < 0) return;
    const int n = sp.t1 - sp.t0, c = tid % LPT;
    unsigned char* const blk = p.pool + (static_cast<size_t>(sp.page) * p.Hk + h) * B::BYTES;
    const T* const kin = static_cast<const T*>(p.k.p) + b * p.k.sb + sp.i0 * p.k.sn + h * p.k.sh + 8 * c;
    const T* const vin = static_cast<const T*>(p.v.p) + b * p.v.sb + sp.i0 * p.v.sn + h * p.v.sh + 8 * c;
    // every thread of a warp takes part in the exchanges, whether or not it has a token
    for (int base = 0; base < 2 * n; base += U * PER) {
        Eight<T> e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * PER + tid / LPT;
            if (i < 2 * n) e[u].load(i < n ? kin + i * p.k.sn : vin + (i - n) * p.v.sn);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * PER + tid / LPT;
            if (base + u * PER >= 2 * n) break;      // the same for every thread
            const bool live = i < 2 * n, val = i >= n;
            const int t = sp.t0 + (val ? i - n : i);
            float x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = 0.f;
            if (live) e[u].get(x);
            float top = 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) top = fmaxf(top, fabsf(x[q]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int sb = scale_bits(__fdiv_rn(top, 7.f));
            const float s = scale_value(sb);
            const uint32_t w = codes_of(x, s > 0.f ? __frcp_rn(s) : 0.f);
            if (live) {
                if (val) s_codes[t][c] = w;
                else *reinterpret_cast<uint32_t*>(blk + B::key(c / 4, t) + (c % 4) * 4) = w;
                if (c % 4 == 0) blk[(val ? B::VS : B::KS) + t * B::NG + c / 4] = static_cast<unsigned char>(sb);
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < 4 * (D / 2); i += TOK_THREADS) {
        const int t = i / (D / 2) * 16, r = i % (D / 2), lo = max(sp.t0 - t, 0), hi = min(sp.t1 - t, 16);
        if (lo >= hi) continue;
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 16; ++q)
            if (q >= lo && q < hi) {
                const uint32_t a = s_codes[t + q][r / 8] >> (r % 8 * 4), z = s_codes[t + q][(r + D / 2) / 8] >> (r % 8 * 4);
                w[q / 4] |= ((a & 15u) | (z & 15u) << 4) << (q % 4 * 8);
            }
        unsigned char* const to = blk + B::value(t, r);
        if (lo == 0 && hi == 16) {
            *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int q = 0; q < 16; ++q)
                if (q >= lo && q < hi) to[q] = static_cast<unsigned char>(w[q / 4] >> (q % 4 * 8));
        }
    }
}

// The reverse: D / 8 lanes write a token, eight channels each. Keys are read where they lie; value codes, 16 tokens of
// two channels at a time, go through shared memory as bytes by token. Positions without a page, outside the table or past
// the count give zeros.
template <class T, int D>
__global__ void __launch_bounds__(TOK_THREADS) read_kernel(const __grid_constant__ TokensParams p) {
    using B = Block<D>;
    constexpr int LPT = D / 8;
    __shared__ __align__(16) unsigned char s_codes[PAGE][D / 2];
    const int h = blockIdx.x, b = blockIdx.z, tid = threadIdx.x, c = tid % LPT;
    Span sp;
    const bool some = span_of(p, b, blockIdx.y, h == 0 && tid == 0, sp), held = some && sp.page >= 0;
    const unsigned char* const blk = p.pool + (static_cast<size_t>(held ? sp.page : 0) * p.Hk + h) * B::BYTES;
    auto put = [&](const Heads& o, long long i, const float (&x)[8]) {
        Eight<T> e;
        e.set(x);
        e.store(static_cast<T*>(o.p) + b * o.sb + i * o.sn + h * o.sh + 8 * c);
    };
    if (held && p.v.p)
        for (int i = tid; i < 4 * (D / 2); i += TOK_THREADS) {
            const int t = i / (D / 2) * 16, r = i % (D / 2);
            if (t + 16 <= sp.t0 || t >= sp.t1) continue;
            const uint4 v = *reinterpret_cast<const uint4*>(blk + B::value(t, r));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 16; ++q) s_codes[t + q][r] = static_cast<unsigned char>(w[q / 4] >> (q % 4 * 8));
        }
    __syncthreads();
    if (some) {
        const int n = sp.t1 - sp.t0;
#pragma unroll 4
        for (int i = tid / LPT; i < n; i += TOK_THREADS / LPT) {
            const int t = sp.t0 + i;
            float x[8];
            if (p.k.p) {
                const uint32_t w = held ? *reinterpret_cast<const uint32_t*>(blk + B::key(c / 4, t) + (c % 4) * 4) : 0u;
                const float s = held ? scale_value(blk[B::KS + t * B::NG + c / 4]) : 0.f;
#pragma unroll
                for (int q = 0; q < 8; ++q) x[q] = held ? static_cast<float>(static_cast<int>((w >> (4 * q)) & 15u) - 8) * s : 0.f;
                put(p.k, sp.i0 + i, x);
            }
            if (p.v.p) {
                const float s = held ? scale_value(blk[B::VS + t * B::NG + c / 4]) : 0.f;
                const int up = 8 * c >= D / 2 ? 4 : 0;
                const uint2 w = *reinterpret_cast<const uint2*>(&s_codes[t][8 * c % (D / 2)]);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    x[q] = held ? static_cast<float>(static_cast<int>(((q < 4 ? w.x : w.y) >> (q % 4 * 8 + up)) & 15u) - 8) * s : 0.f;
                put(p.v, sp.i0 + i, x);
            }
        }
    }
    // inputs that no page of the table covers: CTA y clears its share of them
    const int start = p.start[b];
    const int cnt = min(max(p.counts ? p.counts[b] : p.N, 0), p.N);
    const long long room = static_cast<long long>(p.max_pages) * PAGE, a = static_cast<long long>(blockIdx.y) * PAGE;
    const float zero[8] = {};
    for (int u = tid / LPT; u < PAGE; u += TOK_THREADS / LPT) {
        const long long i = a + u, pos = start + i;
        if (i < p.N && (i >= cnt || pos < 0 || pos >= room)) {
            if (p.k.p) put(p.k, i, zero);
            if (p.v.p) put(p.v, i, zero);
        }
    }
}

}  // namespace specc
