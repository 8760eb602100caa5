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

__device__ __forceinline__ float max3_nan(float a, float b, float c) {      // a NaN if any is
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

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
    const int room = p.max_pages * PAGE;      // below 2^31
    const int lo = max(start, 0), hi = start > room - cnt ? room : start + cnt;
    if ((start < 0 || start > room - cnt) && report) atomicOr(p.status, SPEC_STATUS_BAD_LENGTH);
    const int j = lo / PAGE + y;
    if (j > (hi - 1) / PAGE || hi <= lo) return false;
    s.t0 = max(lo - j * PAGE, 0);
    s.t1 = min(hi - j * PAGE, PAGE);
    s.i0 = j * PAGE + s.t0 - start;
    s.page = p.table[static_cast<size_t>(b) * p.max_pages + j];
    if (s.page < 0 || s.page >= p.pages) {
        if (report) atomicOr(p.status, SPEC_STATUS_BAD_PAGE);
        s.page = -1;
    }
    return true;
}

// One CTA quantises the keys, or the values, of the tokens of one page and head (blockIdx.x: head, then which); no two
// CTAs write a byte of the same token, so pages that start or end inside the call's range need no read. D / 8 lanes take a
// token, four of them a group; a page's loads are all in flight together. Keys go to the page as they come: two tokens of a
// warp fill a sector of each group. A value's codes lie with those of 15 other tokens, so they pass through shared
// memory: there as words of eight channels by token, from there a thread gathers the 16 tokens of a byte row, two
// channels, and writes 16 bytes (or, in a run that the range does not fill, the bytes that are its own).
// 17400 tokens of 8 heads of 128 take 26 us (2.7 TB/s of 71 MB in and 19 MB out): instructions bound it, 79% of the slots are
// taken; 41 us with divisions for the codes and keys and values in one CTA.
template <class T, int D>
__global__ void __launch_bounds__(TOK_THREADS) append_kernel(const __grid_constant__ TokensParams p) {
    using B = Block<D>;
    constexpr int LPT = D / 8, PER = TOK_THREADS / LPT;      // lanes of a token, tokens of a pass
    constexpr int U = PAGE / PER;                            // passes of a page
    __shared__ uint32_t s_codes[PAGE][LPT];
    after_previous();
    const bool val = blockIdx.x >= p.Hk;
    const int h = val ? blockIdx.x - p.Hk : blockIdx.x, b = blockIdx.z, tid = threadIdx.x;
    Span sp;
    if (!span_of(p, b, blockIdx.y, blockIdx.x == 0 && tid == 0, sp) || sp.page < 0) return;
    const int n = sp.t1 - sp.t0, c = tid % LPT;
    const Heads& in = val ? p.v : p.k;
    unsigned char* const blk = p.pool + (static_cast<size_t>(sp.page) * p.Hk + h) * B::BYTES;
    const T* src = static_cast<const T*>(in.p) + b * in.sb + (sp.i0 + tid / LPT) * in.sn + h * in.sh + 8 * c;
    Eight<T> e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        e[u] = {};
        if (u * PER + tid / LPT < n) e[u].load(src);
        src += PER * in.sn;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u * PER >= n) break;      // the same for every thread: all of a warp take part in the exchanges
        const int i = u * PER + tid / LPT, t = sp.t0 + i;
        float x[8], top = 0.f;
        e[u].get(x);
#pragma unroll
        for (int q = 0; q < 8; q += 2) top = max3_nan(top, fabsf(x[q]), fabsf(x[q + 1]));
        if (top != top) {             // a NaN counts as 0
            top = 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                x[q] = x[q] == x[q] ? x[q] : 0.f;
                top = fmaxf(top, fabsf(x[q]));
            }
        }
        __syncwarp();
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int sb = scale_bits(top);
        const float s = scale_value(sb);
        const uint32_t w = sb >= 8 && sb < SCALE_TOP ? codes_of<false>(x, s) : codes_of<true>(x, s);
        if (i < n) {
            if (val) s_codes[t][c] = w;
            else *reinterpret_cast<uint32_t*>(blk + B::key(c / 4, t) + (c % 4) * 4) = w;
            if (c % 4 == 0) blk[(val ? B::VS : B::KS) + t * B::NG + c / 4] = static_cast<unsigned char>(sb);
        }
    }
    if (!val) return;
    __syncthreads();
    for (int i = tid; i < 4 * (D / 2); i += TOK_THREADS) {
        const int t = i / (D / 2) * 16, r = i % (D / 2), lo = max(sp.t0 - t, 0), hi = min(sp.t1 - t, 16);
        if (lo >= hi) continue;
        unsigned char* const to = blk + B::value(t, r);
        auto both = [&](int q) {
            const uint32_t a = s_codes[t + q][r / 8] >> (r % 8 * 4), z = s_codes[t + q][(r + D / 2) / 8] >> (r % 8 * 4);
            return (a & 15u) | (z & 15u) << 4;
        };
        if (lo == 0 && hi == 16) {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 16; ++q) w[q / 4] |= both(q) << (q % 4 * 8);
            *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int q = lo; q < hi; ++q) to[q] = static_cast<unsigned char>(both(q));
        }
    }
}

// The reverse, again keys and values apart: D / 8 lanes write a token, eight channels each. Keys are read where they lie;
// value codes, 16 tokens of two channels at a time, go through shared memory as bytes by token. Positions without a page,
// outside the table or past the count give zeros: CTA y clears those among inputs 64 y ...
// Writes bound it: 32768 tokens, 17400 of them cached, of 8 heads of 128 take 30 us (153 MB, 5 TB/s).
template <class T, int D>
__global__ void __launch_bounds__(TOK_THREADS) read_kernel(const __grid_constant__ TokensParams p) {
    using B = Block<D>;
    constexpr int LPT = D / 8, PER = TOK_THREADS / LPT;
    __shared__ __align__(16) unsigned char s_codes[PAGE][D / 2];
    after_previous();
    const bool val = blockIdx.x >= p.Hk;
    const int h = val ? blockIdx.x - p.Hk : blockIdx.x, b = blockIdx.z, tid = threadIdx.x, c = tid % LPT;
    const Heads& o = val ? p.v : p.k;
    if (!o.p) return;
    Span sp;
    const bool some = span_of(p, b, blockIdx.y, h == 0 && tid == 0, sp), held = some && sp.page >= 0;
    T* const out = static_cast<T*>(o.p) + b * o.sb + h * o.sh + 8 * c;
    if (held) {
        const unsigned char* const blk = p.pool + (static_cast<size_t>(sp.page) * p.Hk + h) * B::BYTES;
        if (val) {
            for (int i = tid; i < 4 * (D / 2); i += TOK_THREADS) {
                const int t = i / (D / 2) * 16, r = i % (D / 2);
                if (t + 16 <= sp.t0 || t >= sp.t1) continue;
                const uint4 v = *reinterpret_cast<const uint4*>(blk + B::value(t, r));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 16; ++q) s_codes[t + q][r] = static_cast<unsigned char>(w[q / 4] >> (q % 4 * 8));
            }
            __syncthreads();
        }
        const int n = sp.t1 - sp.t0;
#pragma unroll 4
        for (int i = tid / LPT; i < n; i += PER) {
            const int t = sp.t0 + i;
            // 0x6400 | c + 8 is the half 1032 + c: less 1032 and times the scale, both exactly
            const uint32_t s = blk[(val ? B::VS : B::KS) + t * B::NG + c / 4] * 0x00800080u;
            uint32_t h[4];
            if (val) {
                const uint2 w = *reinterpret_cast<const uint2*>(&s_codes[t][8 * c % (D / 2)]);
                const int up = 8 * c >= D / 2 ? 4 : 0;
                const uint32_t a = w.x >> up & 0x0F0F0F0Fu, z = w.y >> up & 0x0F0F0F0Fu;
                h[0] = __byte_perm(a, 0x64u, 0x4140), h[1] = __byte_perm(a, 0x64u, 0x4342);
                h[2] = __byte_perm(z, 0x64u, 0x4140), h[3] = __byte_perm(z, 0x64u, 0x4342);
            } else {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + B::key(c / 4, t) + (c % 4) * 4);
                uint32_t g[4];      // codes q and q + 4
#pragma unroll
                for (int q = 0; q < 4; ++q) g[q] = (w >> (4 * q) & 0x000F000Fu) | 0x64006400u;
                h[0] = __byte_perm(g[0], g[1], 0x5410), h[1] = __byte_perm(g[2], g[3], 0x5410);
                h[2] = __byte_perm(g[0], g[1], 0x7632), h[3] = __byte_perm(g[2], g[3], 0x7632);
            }
            float x[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const __half2 v = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&h[q]), __float2half2_rn(1032.f)),
                                          *reinterpret_cast<const __half2*>(&s));
                const float2 f = __half22float2(v);
                x[2 * q] = f.x, x[2 * q + 1] = f.y;
            }
            Eight<T> e;
            e.set(x);
            e.store(out + (sp.i0 + i) * o.sn);
        }
    }
    // inputs without a cached token: those of the page where there is none, and of inputs 64 y .. those before and behind the
    // run [v0, v1) that lies in the table
    const int start = p.start[b], cnt = min(max(p.counts ? p.counts[b] : p.N, 0), p.N);
    const long long room = static_cast<long long>(p.max_pages) * PAGE;
    const int v0 = static_cast<int>(min(max(-static_cast<long long>(start), 0LL), static_cast<long long>(cnt)));
    const int v1 = static_cast<int>(max(min(room - start, static_cast<long long>(cnt)), static_cast<long long>(v0)));
    const float zero[8] = {};
    Eight<T> none;
    none.set(zero);
    auto clear = [&](int from, int to) {
#pragma unroll 4
        for (int i = from + tid / LPT; i < to; i += PER) none.store(out + i * o.sn);
    };
    const int a = blockIdx.y * PAGE, z = min(a + PAGE, p.N);
    if (some && !held) clear(sp.i0, sp.i0 + sp.t1 - sp.t0);
    clear(a, min(z, v0));
    clear(max(a, v1), z);
}

}  // namespace specc
