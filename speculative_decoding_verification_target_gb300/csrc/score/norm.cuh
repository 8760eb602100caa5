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
    int tpr;       // threads of a row: a multiple of 32
    float eps;
    int norm;      // 0: codes of x as it is
};

// The larger magnitude; a NaN stays.
__device__ __forceinline__ float larger(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// 127 p / m is rounded to the nearest integer, ties to even, as if it were exact. The exact product of p and the rounded 127 / m is
// off by 127 x 2^-24 at most, so the integer next to it is the right one unless it lies that near to the middle of two. There the
// exact products decide: with k the integer below, 254 p against (2 k + 1) m, each as a float and its rounding error.
struct Codes {
    float m, by, scale;      // the row's largest magnitude, 127 / m, and the power of two that brings m into range for the exact step
    bool all;                // every code by the exact step
    __device__ explicit Codes(float top) : m(top) {
        scale = top < 8.6736174e-19f ? 1.8446744e19f : top > 1.1529215e18f ? 5.4210109e-20f : 1.f;      // 2^-60: 2^64, 2^60: 2^-64
        all = scale != 1.f && top > 0.f;
        by = top > 0.f ? 127.f / top : 0.f;
    }
    __device__ int exact(float p) const {
        if (m == 0.f) return 0;
        float ps = p * scale, ms = m * scale;
        if (ms < 8.6736174e-19f) ps *= 1.8446744e19f, ms *= 1.8446744e19f;      // the smallest subnormal numbers
        const float k = floorf(ps * (127.f / ms)), h = 2.f * k + 1.f;
        // rounded by themselves: joined with the difference, a product would count its rounding error twice
        const float a = __fmul_rn(254.f, ps), b = __fmul_rn(h, ms);
        const float d = __fadd_rn(__fsub_rn(a, b), __fsub_rn(fmaf(254.f, ps, -a), fmaf(h, ms, -b)));
        const bool up = d > 0.f || (d == 0.f && (static_cast<int>(k) & 1));
        return static_cast<int>(k) + (up ? 1 : 0);
    }
    // Codes of n values; the low byte of each float's bits in c.
    static constexpr float DOUBT = 0.49999f;
    template <int n>
    __device__ void of(const float (&p)[n], uint32_t (&c)[n]) const {
        float off = all ? 1.f : 0.f;
        if constexpr (n % 2 == 0) {
            const unsigned long long by2 = specc::pack2(by, by), magic = specc::pack2(12582912.f, 12582912.f), minus = specc::pack2(-1.f, -1.f);
#pragma unroll
            for (int i = 0; i < n; i += 2) {
                const unsigned long long v = specc::pack2(p[i], p[i + 1]), f = specc::fma2(v, by2, magic);      // its last place is 1
                const float2 d = specc::unpack2(specc::fma2(v, by2, specc::fma2(f, minus, magic))), c2 = specc::unpack2(f);
                off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
                c[i] = __float_as_uint(c2.x), c[i + 1] = __float_as_uint(c2.y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float f = fmaf(p[i], by, 12582912.f);
                off = fmaxf(off, fabsf(fmaf(p[i], by, 12582912.f - f)));
                c[i] = __float_as_uint(f);
            }
        }
        if (off > DOUBT) {      // one after the other, by choosing among the registers: a copy of the step for each made it no faster
            unsigned left = 0u;
#pragma unroll
            for (int i = 0; i < n; ++i)
                left |= (all || fabsf(fmaf(p[i], by, 12582912.f - __uint_as_float(c[i]))) > DOUBT ? 1u : 0u) << i;
            for (; left; left &= left - 1) {
                const int at = __ffs(left) - 1;
                float v = p[0];
#pragma unroll
                for (int i = 1; i < n; ++i) v = i == at ? p[i] : v;
                const uint32_t e = static_cast<uint32_t>(exact(v));
#pragma unroll
                for (int i = 0; i < n; ++i) c[i] = i == at ? e : c[i];
            }
        }
    }
};

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// A piece of a row: 16 bytes of values where the rows allow it, else one value.
template <class T, bool VEC>
struct Piece {
    static constexpr int E = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
    using Raw = std::conditional_t<VEC, uint4, T>;
    static __device__ void get(const Raw& r, float (&v)[E]) {
        if constexpr (!VEC) v[0] = to_float(r);
        else if constexpr (std::is_same_v<T, float>) {
            v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
        } else {
            specc::Eight<T> e;
            e.r = r;
            e.get(v);
        }
    }
    static __device__ Raw put(const float (&v)[E]) {
        if constexpr (!VEC) return from_float<T>(v[0]);
        else if constexpr (std::is_same_v<T, float>)
            return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        else {
            specc::Eight<T> e;
            e.set(v);
            return e.r;
        }
    }
    static __device__ void codes(signed char* to, const uint32_t (&c)[E]) {
        if constexpr (E == 1) *to = static_cast<signed char>(c[0]);
        else if constexpr (E == 4) *reinterpret_cast<uint32_t*>(to) = pack4(c[0], c[1], c[2], c[3]);
        else *reinterpret_cast<uint2*>(to) = make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
    }
};

// The larger magnitudes of pairs of 16-bit values, as integers: a NaN is above all.
__device__ __forceinline__ uint32_t larger2(uint32_t a, const uint4& x) {
    a = __vmaxu2(a, __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu));
    return __vmaxu2(a, __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
}

// The sum and the largest magnitude over a row's `warps` warps, the first of which is `from`; `turn` alternates.
__device__ __forceinline__ void join_row(float& sum, float& top, int from, int warps, int turn, float2 (*s_part)[32]) {
    sum = specv::warp_sum(sum);
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));      // not negative; a NaN is the largest
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0) s_part[turn][threadIdx.x >> 5] = make_float2(sum, top);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const float2 v = lane < warps ? s_part[turn][from + lane] : make_float2(0.f, 0.f);
    sum = specv::warp_sum(v.x);
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v.y)));
}

// A row is in the registers of tpr threads, SLOTS pieces each, between its one read and its one write; the next row of these
// threads is on its way meanwhile, and the weights stay. Bandwidth bounds many rows, latency few: there a row has more threads.
// FULL: with a residual, a weight or a norm; else codes of the rows as they are, with half the registers. 16384 rows of 4096 in bf16,
// with all of it, take 78.8 us (89% of the copy rate), 8192 rows of 14336 as they are 79.6 us (66%; instruction issue, at 16.9 a value, and
// the row's barrier). With four pieces to codes, bf16's 128 registers spill 24 bytes, and 16-bit types' 64 without a norm 32.
template <class T, bool CODES, int SLOTS, bool VEC, bool FULL>
__global__ void __launch_bounds__(512, FULL ? 1 : 2) norm_rows_kernel(const __grid_constant__ NormParams p) {
    using P = Piece<T, VEC>;
    using Raw = typename P::Raw;
    constexpr int E = P::E;
    __shared__ float2 s_part[2][32];
    after_previous();
    const int per = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr, c = threadIdx.x - sub * p.tpr, pieces = (p.D + E - 1) / E;
    const bool with = FULL && p.res.p != nullptr, weighted = FULL && p.weight != nullptr;
    Raw x[SLOTS], y[SLOTS], w[SLOTS];
    auto place = [&](const Rows& t, long long row) {
        const int b = static_cast<int>(row / p.N), n = static_cast<int>(row - static_cast<long long>(b) * p.N);
        return b * t.sb + n * t.sn;
    };
    auto fetch = [&](long long row) {
        if (row >= p.rows) return;
        const T* const px = static_cast<const T*>(p.x.p) + place(p.x, row);
        const T* const py = with ? static_cast<const T*>(p.res.p) + place(p.res, row) : px;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (c + s * p.tpr < pieces) {
                x[s] = *reinterpret_cast<const Raw*>(px + (c + s * p.tpr) * E);
                if (with) y[s] = *reinterpret_cast<const Raw*>(py + (c + s * p.tpr) * E);
            }
    };
    long long row = static_cast<long long>(blockIdx.x) * per + sub;
    fetch(row);
    if (weighted) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (c + s * p.tpr < pieces) w[s] = *reinterpret_cast<const Raw*>(static_cast<const T*>(p.weight) + (c + s * p.tpr) * E);
    }
    const long long step = static_cast<long long>(gridDim.x) * per;
    int turn = 0;
    for (long long base = row - sub; base < p.rows; base += step, row += step, turn ^= 1) {
        constexpr bool AS_IS = !FULL && VEC && sizeof(T) == 2;      // kept as they were read
        std::conditional_t<AS_IS, Raw, float[E]> r[SLOTS];
        float sum = 0.f, top = 0.f;
        uint32_t pairs = 0u;
        T* const res_out = with && row < p.rows ? static_cast<T*>(p.res_out.p) + place(p.res_out, row) : nullptr;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            if (row >= p.rows || c + s * p.tpr >= pieces) continue;
            if constexpr (AS_IS) {
                r[s] = x[s];
                pairs = larger2(pairs, x[s]);
                continue;
            } else {
            P::get(x[s], r[s]);
            if (with) {
                float add[E];
                P::get(y[s], add);
#pragma unroll
                for (int i = 0; i < E; ++i) r[s][i] += add[i];
                const Raw rounded = P::put(r[s]);
                *reinterpret_cast<Raw*>(res_out + (c + s * p.tpr) * E) = rounded;
                P::get(rounded, r[s]);
            }
            float g[E];
            if (weighted) P::get(w[s], g);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (FULL) sum = fmaf(r[s][i], r[s][i], sum);
                if (weighted) r[s][i] *= g[i];
                if (CODES) top = larger(top, r[s][i]);
            }
            }
        }
        if constexpr (AS_IS) {
            const unsigned short m = static_cast<unsigned short>(max(pairs & 0xFFFFu, pairs >> 16));
            if constexpr (std::is_same_v<T, __half>) top = __half2float(__ushort_as_half(m));
            else top = __uint_as_float(static_cast<uint32_t>(m) << 16);
        }
        fetch(row + step);
        join_row(sum, top, threadIdx.x / 32 - c / 32, p.tpr / 32, turn, s_part);
        if (row >= p.rows) continue;
        const float inv = FULL && p.norm ? rsqrtf(sum / p.D + p.eps) : 1.f;
        if constexpr (CODES) {
            const bool bad = !(top < INFINITY);
            const Codes codes(bad ? 0.f : top);
            signed char* const out = static_cast<signed char*>(p.out.p) + place(p.out, row);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                if (c + s * p.tpr >= pieces) continue;
                uint32_t q[E];
                float v[E];
                if constexpr (AS_IS) P::get(r[s], v);
                else {
#pragma unroll
                    for (int i = 0; i < E; ++i) v[i] = r[s][i];
                }
                if (bad) {
#pragma unroll
                    for (int i = 0; i < E; ++i) v[i] = 0.f;
                }
                codes.of(v, q);
                P::codes(out + (c + s * p.tpr) * E, q);
            }
            if (c == 0) p.scale[row] = bad ? NAN : top / 127.f * inv;
        } else if constexpr (!AS_IS) {
            T* const out = static_cast<T*>(p.out.p) + place(p.out, row);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                if (c + s * p.tpr >= pieces) continue;
#pragma unroll
                for (int i = 0; i < E; ++i) r[s][i] *= inv;
                *reinterpret_cast<Raw*>(out + (c + s * p.tpr) * E) = P::put(r[s]);
            }
        }
    }
}

// 16-bit rows of which each begins elsewhere within 16 bytes, but all of a token's alike, as those of an odd width do: pieces of 16
// bytes from the row's first such place on, and up to seven single values at either end, one a thread. The weights come from shared
// memory, shifted by the row's place. 5001 rows of 2051 in fp16 take 22.7 us on the device (value by value 27.6), 8192 rows of 4099 in bf16
// 60.0 us, to codes, which are stored byte by byte, 70.7 (floors 40.2 and 35.2).
template <class T, bool CODES, int SLOTS>
__global__ void __launch_bounds__(512) norm_peel_kernel(const __grid_constant__ NormParams p) {
    using P = Piece<T, true>;
    constexpr int E = P::E;
    extern __shared__ uint4 s_weight[];      // up to the second piece behind the last value
    __shared__ float2 s_part[2][32];
    after_previous();
    const int per = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr, c = threadIdx.x - sub * p.tpr;
    const bool with = p.res.p != nullptr;
    uint4 x[SLOTS], y[SLOTS];
    T x1 = from_float<T>(0.f), y1 = from_float<T>(0.f);
    auto place = [&](const Rows& t, long long row) {
        const int b = static_cast<int>(row / p.N), n = static_cast<int>(row - static_cast<long long>(b) * p.N);
        return static_cast<T*>(t.p) + b * t.sb + n * t.sn;
    };
    // a row's first value on 16 bytes, its pieces, and the single value that is this thread's or -1
    struct Cut {
        int head, whole, single;
        __device__ Cut(const T* row, int D, int c, int tpr) {
            head = min(D, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / static_cast<int>(sizeof(T)));
            whole = (D - head) / E;
            const int tail = D - head - whole * E, back = tpr - 1 - c;
            single = c < head ? c : back < tail ? D - 1 - back : -1;
        }
    };
    auto fetch = [&](long long row) {
        if (row >= p.rows) return;
        const T *const px = place(p.x, row), *const py = with ? place(p.res, row) : px;
        const Cut cut(px, p.D, c, p.tpr);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (c + s * p.tpr < cut.whole) {
                x[s] = *reinterpret_cast<const uint4*>(px + cut.head + (c + s * p.tpr) * E);
                if (with) y[s] = *reinterpret_cast<const uint4*>(py + cut.head + (c + s * p.tpr) * E);
            }
        if (cut.single >= 0) {
            x1 = px[cut.single];
            if (with) y1 = py[cut.single];
        }
    };
    long long row = static_cast<long long>(blockIdx.x) * per + sub;
    fetch(row);
    const T* const w = static_cast<const T*>(p.weight);
    T* const sw = reinterpret_cast<T*>(s_weight);
    if (w) {
        for (int i = threadIdx.x; i < (p.D + 7) / 8 * 8 + 8; i += blockDim.x) sw[i] = i < p.D ? w[i] : from_float<T>(0.f);
        __syncthreads();
    }
    const long long step = static_cast<long long>(gridDim.x) * per;
    int turn = 0;
    for (long long base = row - sub; base < p.rows; base += step, row += step, turn ^= 1) {
        const bool real = row < p.rows;
        const Cut cut(real ? place(p.x, row) : nullptr, p.D, c, p.tpr);
        T* const res_out = with && real ? place(p.res_out, row) : nullptr;
        float r[SLOTS][E], r1 = 0.f, sum = 0.f, top = 0.f;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int q = c + s * p.tpr;
            if (!real || q >= cut.whole) continue;
            P::get(x[s], r[s]);
            if (with) {
                float add[E];
                P::get(y[s], add);
#pragma unroll
                for (int i = 0; i < E; ++i) r[s][i] += add[i];
                const uint4 rounded = P::put(r[s]);
                *reinterpret_cast<uint4*>(res_out + cut.head + q * E) = rounded;
                P::get(rounded, r[s]);
            }
            float g[E];
            if (w) {
                const uint4 a = s_weight[q], b = s_weight[q + 1];
                const uint32_t t[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                const int by = cut.head >> 1;
                uint32_t m[5], u[4];
#pragma unroll
                for (int i = 0; i < 5; ++i) m[i] = by == 0 ? t[i] : by == 1 ? t[i + 1] : by == 2 ? t[i + 2] : t[i + 3];
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = cut.head & 1 ? __byte_perm(m[i], m[i + 1], 0x5432) : m[i];
                P::get(make_uint4(u[0], u[1], u[2], u[3]), g);
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                sum = fmaf(r[s][i], r[s][i], sum);
                if (w) r[s][i] *= g[i];
                if (CODES) top = larger(top, r[s][i]);
            }
        }
        if (real && cut.single >= 0) {
            r1 = to_float(x1);
            if (with) {
                const T rounded = from_float<T>(r1 + to_float(y1));
                res_out[cut.single] = rounded;
                r1 = to_float(rounded);
            }
            sum = fmaf(r1, r1, sum);
            if (w) r1 *= to_float(sw[cut.single]);
            if (CODES) top = larger(top, r1);
        }
        fetch(row + step);
        join_row(sum, top, threadIdx.x / 32 - c / 32, p.tpr / 32, turn, s_part);
        if (!real) continue;
        const float inv = p.norm ? rsqrtf(sum / p.D + p.eps) : 1.f;
        if constexpr (CODES) {
            const bool bad = !(top < INFINITY);
            const Codes codes(bad ? 0.f : top);
            const int b = static_cast<int>(row / p.N), n = static_cast<int>(row - static_cast<long long>(b) * p.N);
            signed char* const out = row_of<signed char>(p.out, b, n);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                const int q = c + s * p.tpr;
                if (q >= cut.whole) continue;
                uint32_t k[E];
                if (bad) {
#pragma unroll
                    for (int i = 0; i < E; ++i) r[s][i] = 0.f;
                }
                codes.of(r[s], k);
#pragma unroll
                for (int i = 0; i < E; ++i) out[cut.head + q * E + i] = static_cast<signed char>(k[i]);
            }
            if (cut.single >= 0) {
                const float one[1] = {bad ? 0.f : r1};
                uint32_t k[1];
                codes.of(one, k);
                out[cut.single] = static_cast<signed char>(k[0]);
            }
            if (c == 0) p.scale[row] = bad ? NAN : top / 127.f * inv;
        } else {
            T* const out = place(p.out, row);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                const int q = c + s * p.tpr;
                if (q >= cut.whole) continue;
#pragma unroll
                for (int i = 0; i < E; ++i) r[s][i] *= inv;
                *reinterpret_cast<uint4*>(out + cut.head + q * E) = P::put(r[s]);
            }
            if (cut.single >= 0) out[cut.single] = from_float<T>(r1 * inv);
        }
    }
}

// Rows that do not fit in registers: read twice, the second time from the caches, a value a load. 2048 fp32 rows of 16384 to codes take
// 116.5 us, 1024 bf16 rows of 32768 110 us (floors 65.2 and 35.1).
template <class T, bool CODES>
__global__ void __launch_bounds__(512) norm_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 s_part[2][32];
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
    float sum = 0.f, top = 0.f;
    for (int i = threadIdx.x; i < p.D; i += 512) {
        const float r = value(i);
        sum = fmaf(r, r, sum);
        top = larger(top, w ? r * to_float(w[i]) : r);
    }
    join_row(sum, top, 0, 16, 0, s_part);
    const float inv = p.norm ? rsqrtf(sum / p.D + p.eps) : 1.f;
    const bool bad = !(top < INFINITY);
    const Codes codes(bad ? 0.f : top);
    for (int i = threadIdx.x; i < p.D; i += 512) {
        const float r = value(i), q[1] = {w ? r * to_float(w[i]) : r};
        if (res) row_of<T>(p.res_out, b, n)[i] = from_float<T>(r);
        if (CODES) {
            uint32_t c[1] = {0u};
            if (!bad) codes.of(q, c);
            row_of<signed char>(p.out, b, n)[i] = static_cast<signed char>(c[0]);
        } else {
            row_of<T>(p.out, b, n)[i] = from_float<T>(q[0] * inv);
        }
    }
    if (CODES && threadIdx.x == 0) p.scale[t] = bad ? NAN : top / 127.f * inv;
}

}  // namespace specs
