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

// The bytes of a block's token range [t0, t1), moved between shared and global memory: key codes as 16 bytes a
// token and group, value codes as 16 bytes a channel pair where the whole run of 16 tokens is in the range and
// byte by byte where it is not, scales byte by byte (runs of neighbouring threads).
template <int D, bool STORE>
__device__ __forceinline__ void move_block(unsigned char* g, unsigned char* s, int t0, int t1, int tid) {
    using B = Block<D>;
    const int n = t1 - t0;
    for (int i = tid; i < B::NG * n; i += TOK_THREADS) {
        const int o = B::key(i / n, t0 + i % n);
        if (STORE) *reinterpret_cast<uint4*>(g + o) = *reinterpret_cast<const uint4*>(s + o);
        else *reinterpret_cast<uint4*>(s + o) = *reinterpret_cast<const uint4*>(g + o);
    }
    for (int i = tid; i < B::NG * n; i += TOK_THREADS) {
        const int o = t0 * B::NG + i;
        if (STORE) g[B::KS + o] = s[B::KS + o], g[B::VS + o] = s[B::VS + o];
        else s[B::KS + o] = g[B::KS + o], s[B::VS + o] = g[B::VS + o];
    }
    for (int run = t0 / 16; run * 16 < t1; ++run) {
        if (!STORE || (run * 16 >= t0 && run * 16 + 16 <= t1)) {
            for (int r = tid; r < D / 2; r += TOK_THREADS) {
                const int o = B::value(run * 16, r);
                if (STORE) *reinterpret_cast<uint4*>(g + o) = *reinterpret_cast<const uint4*>(s + o);
                else *reinterpret_cast<uint4*>(s + o) = *reinterpret_cast<const uint4*>(g + o);
            }
        } else {
            const int a = max(t0, run * 16), z = min(t1, run * 16 + 16), m = z - a;
            for (int i = tid; i < m * (D / 2); i += TOK_THREADS) {
                const int o = B::value(a + i % m, i / m);
                g[o] = s[o];
            }
        }
    }
}

// One CTA quantises the tokens of one page and head into a block in shared memory, laid out as in the pool, and
// then writes the part that it filled; no two CTAs write a byte of the same token, so pages that start or end
// inside the call's range need no read. D / 8 lanes take a token, four of them a group.
template <class T, int D>
__global__ void __launch_bounds__(TOK_THREADS) append_kernel(const __grid_constant__ TokensParams p) {
    using B = Block<D>;
    constexpr int LPT = D / 8;
    __shared__ __align__(16) unsigned char s_blk[B::BYTES];
    const int h = blockIdx.x, b = blockIdx.z, tid = threadIdx.x;
    Span sp;
    if (!span_of(p, b, blockIdx.y, h == 0 && tid == 0, sp) || sp.page < 0) return;
    const int n = sp.t1 - sp.t0, c = tid % LPT, lane = tid & 31;
    // every thread of a warp takes part in the exchanges, whether or not it has a token
    for (int base = 0; base < 2 * n; base += TOK_THREADS / LPT) {
        const int u = base + tid / LPT;
        const bool live = u < 2 * n, val = u >= n;
        const int t = sp.t0 + (val ? u - n : u);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
        if (live) {
            const Heads& in = val ? p.v : p.k;
            Eight<T> e;
            e.load(static_cast<const T*>(in.p) + b * in.sb + static_cast<long long>(sp.i0 + t - sp.t0) * in.sn + h * in.sh +
                   8 * c);
            e.get(x);
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int sb = scale_bits(__fdiv_rn(top, 7.f));
        const float s = scale_value(sb);
        uint32_t w = 0;   // eight codes, the i-th in bits 4 i
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= code_of(x[i], s) << (4 * i);
        const uint32_t up = __shfl_sync(0xffffffffu, w, (lane + LPT / 2) & 31);   // of the channels D / 2 further on
        if (live) {
            if (!val) {
                *reinterpret_cast<uint32_t*>(s_blk + B::key(c / 4, t) + (c % 4) * 4) = w;
                if (c % 4 == 0) s_blk[B::KS + t * B::NG + c / 4] = static_cast<unsigned char>(sb);
            } else {
                if (c < LPT / 2) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        s_blk[B::value(t, 8 * c + i)] =
                            static_cast<unsigned char>(((w >> (4 * i)) & 15u) | (((up >> (4 * i)) & 15u) << 4));
                }
                if (c % 4 == 0) s_blk[B::VS + t * B::NG + c / 4] = static_cast<unsigned char>(sb);
            }
        }
    }
    __syncthreads();
    unsigned char* const g = p.pool + (static_cast<size_t>(sp.page) * p.Hk + h) * B::BYTES;
    move_block<D, true>(g, s_blk, sp.t0, sp.t1, tid);
}

// The reverse: a block's token range into shared memory, then each thread writes eight channels of a token.
// Positions without a page, outside the table or past the count give zeros: grid y covers all N inputs of a
// sequence in runs of 64 that need not be the pages' own.
template <class T, int D>
__global__ void __launch_bounds__(TOK_THREADS) read_kernel(const __grid_constant__ TokensParams p) {
    using B = Block<D>;
    constexpr int LPT = D / 8;
    __shared__ __align__(16) unsigned char s_blk[B::BYTES];
    const int h = blockIdx.x, b = blockIdx.z, tid = threadIdx.x;
    Span sp;
    const bool some = span_of(p, b, blockIdx.y, h == 0 && tid == 0, sp);
    if (some && sp.page >= 0) {
        unsigned char* const g = p.pool + (static_cast<size_t>(sp.page) * p.Hk + h) * B::BYTES;
        move_block<D, false>(g, s_blk, sp.t0, sp.t1, tid);
    }
    __syncthreads();
    auto put = [&](const Heads& o, int i, int c, const float (&x)[8]) {
        Eight<T> e;
        e.set(x);
        e.store(static_cast<T*>(o.p) + b * o.sb + static_cast<long long>(i) * o.sn + h * o.sh + 8 * c);
    };
    if (some) {
        const int n = sp.t1 - sp.t0;
        for (int i = tid; i < n * LPT; i += TOK_THREADS) {
            const int t = sp.t0 + i / LPT, c = i % LPT;
            float x[8];
            if (p.k.p) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(s_blk + B::key(c / 4, t) + (c % 4) * 4);
                const float s = scale_value(s_blk[B::KS + t * B::NG + c / 4]);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    x[q] = sp.page < 0 ? 0.f : static_cast<float>(static_cast<int>((w >> (4 * q)) & 15u) - 8) * s;
                put(p.k, sp.i0 + t - sp.t0, c, x);
            }
            if (p.v.p) {
                const float s = scale_value(s_blk[B::VS + t * B::NG + c / 4]);
                const int r = (8 * c) % (D / 2), sh = 8 * c >= D / 2 ? 4 : 0;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    x[q] = sp.page < 0 ? 0.f : static_cast<float>(static_cast<int>((s_blk[B::value(t, r + q)] >> sh) & 15) - 8) * s;
                put(p.v, sp.i0 + t - sp.t0, c, x);
            }
        }
    }
    // inputs that no page of the table covers: CTA y clears its share of them
    const int start = p.start[b];
    const int cnt = min(max(p.counts ? p.counts[b] : p.N, 0), p.N);
    const long long room = static_cast<long long>(p.max_pages) * PAGE;
    float zero[8] = {};
    const long long a = static_cast<long long>(blockIdx.y) * PAGE;
    for (int u = tid; u < PAGE * LPT; u += TOK_THREADS) {
        const long long i = a + u / LPT, pos = start + i;
        if (i < p.N && (i >= cnt || pos < 0 || pos >= room)) {
            if (p.k.p) put(p.k, static_cast<int>(i), u % LPT, zero);
            if (p.v.p) put(p.v, static_cast<int>(i), u % LPT, zero);
        }
    }
}

}  // namespace specc
