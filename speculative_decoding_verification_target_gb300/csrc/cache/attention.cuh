// Attention of the newest tokens over the 4-bit cache.
//
// For a sequence, a key head and up to NC of the queries that read it (the query heads of the group times the new
// tokens), with keys k_t = c_t s_t and values likewise:
//   S[t, n] = k_t . q_n,  p[t, n] = 2^(S c_n - m_n),  O[d, n] = sum_t v[t, d] p[t, n],  l_n = sum_t p[t, n],  out = O / l.
// Both products run on the 5th-generation tensor cores with the CACHE as the M side: M = 128 tokens for S, M = 128
// channels for O, N = NC queries. So the cost of a tile grows with the queries there are (NC = 16, 32, 48 or 64) and not with
// a padded block of them. The M operand comes from tensor memory, which is what makes 4 bits cheap: a thread is a lane of
// it, turns its own token's (or channel's) codes into halves in registers and stores them there. Neither operand's 16-bit
// form passes through shared memory; that would take three times the bandwidth of the codes themselves, more than shared
// memory has at the rate HBM delivers them.
//   - Codes to halves: one logic and one multiply-add instruction for two, exactly (half_code), and a shift for every
//     second pair; a value code, whose scale changes from code to code, takes one instruction more a pair.
//   - Key codes lie so that a token's 16 bytes of a group are one conflict-free load; the order of channels that
//     falls out, 0 4 1 5 2 6 3 7 in each eight, is given to the queries as well. Value bytes hold channels r and r + D / 2
//     of one token, so that a token can be appended without touching its neighbours' bytes; lanes of the lower
//     and the upper half read the same bytes. Their tokens fall out in the order 0 2 1 3 in each four, which the
//     probabilities' rows follow. A lane's scales change from token to token but are the same for the 32 channels of a
//     warp: a table of them, rebuilt per tile, is read as broadcasts (scales alone, 8 bytes for four tokens: with their
//     offsets beside them it took 195 us where it takes 182, since broadcasts cost shared memory by their bytes). Tokens that
//     hold nothing have s = 0 there, so that whatever bits they have cannot reach O (0 times a NaN would).
//   - The softmax works on S^T: a thread has one token and all queries. m_n is not the maximum but a reference that
//     any value near it may serve as: it is moved, and O and l rescaled, only where a score exceeds it by more than 2^15,
//     which the barrier before the second product detects at no cost. l_n is kept per thread and added up at the end.
//     Probabilities are rounded to fp16 for the product, l is the sum of the unrounded ones. The reference is put 2^-7 of the
//     maximum, so that they take a half's whole range: the largest are 2^7 .. 2^15, all down to 2^-21 of the largest keep their
//     eleven bits, and what is lost of one below that is 2^-32 of the largest at most. (With the reference at the maximum it
//     was 2^-25: beside a first token that takes nearly all the weight, 10^5 others with 2^-25 of it each came to nothing.)
// A tile is 128 tokens, two pages, fetched as one bulk copy each, STAGES tiles ahead, by a warp that also issues the products:
// with that in the computing warps, everyone waited for the one that did it. CTAs are small (four computing warps and four CTAs
// to an SM, as many as the tensor memory has columns for; three CTAs for 25 to 32 queries, whose registers leave room for no
// more; eight warps and two CTAs for over 32) and hide a part of each other's waits.
// Work is split evenly whatever the lengths: the tiles of all (sequence, key head, query block) units form one line, with
// ATT_UNIT places more for each unit's beginning and end, of which each CTA takes an equal run (places of 0, 1, 2, 3 and 4
// tiles: 75, 64, 65, 66 and 67 us on 48 sequences of 130 to 8191 tokens, 74, 66, 63, 62 and 63 us on 96 windows). A unit that is
// cut leaves partial (O, m, l) in the workspace, and a second kernel joins them in a fixed order.
// Measured, 8 key heads of 128: 48 sequences, one query row of four heads each, 219 MB of cache: 61 us, 3.6 TB/s; 64 sequences,
// 24 rows, 627 MB: 180 us, 3.5 TB/s, half of the copy rate. What bounds it: waits within a tile. No unit is full (issue 64% of
// the slots, integer pipe 49%, shared memory 48%, tensor pipe 16%, DRAM 39%): a tile is one chain of codes, product, softmax and
// product in which a CTA's computing warps meet three times, and four warps a scheduler do not cover it (per issued
// instruction fixed latencies 1.25 cycles, barriers 1.11). The 3900 (24 rows) instructions of a tile alone would take
// 975 cycles of four full schedulers, where HBM delivers one in 765; the 3240 of single tokens 810.
#pragma once
#include "cache_format.cuh"
#include "tmem.cuh"

namespace specc {

constexpr int ATT_MAX_CTAS = 640;
constexpr uint64_t ATT_WAIT_NS = 2000000000ull;      // after which a wait gives up
constexpr int ATT_UNIT = 2;             // what beginning and ending a unit costs, in tiles
constexpr float ATT_NONE = -1e30f;       // reference of a query that has seen nothing yet
constexpr float ATT_BELOW = 7.f;         // how far (log2) below the maximum a reference is put
constexpr float ATT_SLACK = 15.f;        // how far (log2) a score may pass the reference: p <= 2^15 is inside a half

struct AttnParams {
    Heads q, out;
    const unsigned char* pool;
    const int* table;
    const int *kv_len, *q_len;
    float* lse;
    unsigned* status;
    int4* desc;              // per CTA: the cut unit that starts in it: sequence, head RB + block, parts (0: none)
    float2* part_ml;         // [2 CTAs][width] (reference, sum)
    float* part_o;           // [2 CTAs][width][D]
    int pages, max_pages, B, N, Hq, Hk, G, window, sinks;
    int RB, rpb;             // query blocks and rows of each
    int width, fp16;         // queries of a part in the workspace; activations in fp16 (else bf16)
    float scale;             // times log2 e
};

// WG warpgroups share a tile's tokens, each with NW of the queries.
template <int D, int WG_, int NW_>
struct Att {
    static constexpr int WG = WG_, NW = NW_;
    static constexpr int CTAS = WG == 2 ? 2 : NW <= 24 ? 4 : 3;      // on an SM, as registers allow
    static constexpr int CT = 128 * WG, TH = CT + 32;     // computing threads; one more warp fetches and issues products
    static constexpr int NQ = WG * NW, NC = (NQ + 15) / 16 * 16;     // queries, and the products' width for them
    static constexpr int TILE = 2 * Block<D>::BYTES;
    // tiles on their way; more gains nothing (72 rows, heads of 128: 389 us with two, 397 with three; heads of 64, 24 rows: 57.0,
    // 56.5 and 57.2 us with two, three and four)
    static constexpr int STAGES = D == 64 || CTAS == 3 ? 3 : 2, INFOS = 2 * STAGES;
    // the second product: D = 128, 128 channels by 128 tokens; D = 64, both pages' channels as 128 rows by 64 tokens, each
    // page's probabilities in columns of their own (half of the result is of no use, but all warps have values to convert)
    static constexpr int ON = D == 128 ? NC : 2 * NC, OK = D == 128 ? 128 : 64;
    static constexpr int WORDS = OK / 4 / WG;             // a thread's words of value codes, four tokens each
    static constexpr int VP = WORDS > 16 ? 2 : 1, WPP = WORDS / VP;
    static constexpr int KQ = NC / 8 * 128, KP = ON / 8 * 128;   // bytes between runs of eight along K, both N operands
    static constexpr int P = STAGES * TILE;               // byte offsets in dynamic shared memory
    static constexpr int Q = P + OK * ON * 2;
    static constexpr int VS = Q + NC * D * 2;
    static constexpr int END = VS + CT / 32 * WORDS * 8;
    // no more CTAs on an SM than its tensor memory has columns for: a further one would wait for one to end
    static constexpr int FLOOR = CTAS == 2 ? 78848 : CTAS == 3 ? 59392 : 47104;
    static constexpr int SMEM = END > FLOOR ? END : FLOOR;
    static constexpr int COL_S = D / 2, COL_O = COL_S + NC;      // tensor memory: operand, S, O
    static constexpr int COLS = WG == 1 ? 128 : 256;
    static_assert(COL_O + ON <= COLS && COLS * CTAS <= 512, "tensor memory");
};

// A sequence's visible pages: [0, a) and [w0, ...), np in all, two to a tile.
struct Seq {
    int len, ql, a, w0, np, T;
};
__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b, bool report) {
    Seq s;
    s.ql = p.q_len ? p.q_len[b] : p.N;
    s.len = p.kv_len[b];
    const int room = p.max_pages * PAGE;
    if (report && (s.ql < 0 || s.ql > p.N || s.len < 0 || s.len > room)) atomicOr(p.status, SPEC_STATUS_BAD_LENGTH);
    s.ql = min(max(s.ql, 0), p.N);
    s.len = min(max(s.len, 0), room);
    s.a = s.w0 = 0;
    if (p.window > 0) {
        const long long first = static_cast<long long>(s.len) - s.ql - p.window + 1;
        s.w0 = first > 0 ? static_cast<int>(first / PAGE) : 0;
        s.a = min(static_cast<int>((static_cast<long long>(p.sinks) + PAGE - 1) / PAGE), s.w0);
    }
    s.np = s.ql > 0 ? s.a + (s.len + PAGE - 1) / PAGE - s.w0 : 0;
    s.T = max(1, (s.np + 1) / 2);        // one empty tile for a unit that sees nothing: it writes its zeros
    return s;
}

// A place in the line of tiles.
struct Cursor {
    int b, h, rb, t;
    Seq s;
    __device__ void next(const AttnParams& p) {
        if (++t < s.T) return;
        t = 0;
        if (++rb < p.RB) return;
        rb = 0;
        if (++h < p.Hk) return;
        h = 0;
        if (++b < p.B) s = load_seq(p, b, false);
    }
    __device__ int page_index(int i) const {      // of the tile's page i, or -1
        const int v = 2 * t + i;
        return v >= s.np ? -1 : v < s.a ? v : s.w0 + v - s.a;
    }
};

// Sums (or maxima) of each of v[0 .. W) over the warp's lanes, to out[0 .. W). Halving exchanges, 31 shuffles for 32
// columns: 32, 16 or 8 at a time.
template <int W, class Op>
__device__ __forceinline__ void fold_columns(float (&v)[W], int lane, float* out, Op op) {
    constexpr int B = W >= 32 ? 32 : W >= 16 ? 16 : 8;
#pragma unroll
    for (int o = B / 2; o > 0; o >>= 1) {
#pragma unroll
        for (int k = 0; k < o; ++k) {
            const bool up = lane & o;
            const float keep = up ? v[k + o] : v[k], send = up ? v[k] : v[k + o];
            v[k] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
#pragma unroll
    for (int o = B; o < 32; o <<= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    if (lane < B) out[lane] = v[0];
    if constexpr (W > B) {
        float rest[W - B];
#pragma unroll
        for (int k = 0; k < W - B; ++k) rest[k] = v[B + k];
        fold_columns(rest, lane, out + B, op);
    }
}

// W columns of this thread's lane: 8, 16, 24 or 32.
template <int W>
__device__ __forceinline__ void tmem_load(uint32_t a, uint32_t (&v)[W]) {
    constexpr int B = W >= 32 ? 32 : W >= 16 ? 16 : 8;
    uint32_t part[B];
    tmem_ld(a, part);
#pragma unroll
    for (int k = 0; k < B; ++k) v[k] = part[k];
    if constexpr (W > B) {
        uint32_t rest[W - B];
        tmem_load<W - B>(a + B, rest);
#pragma unroll
        for (int k = 0; k < W - B; ++k) v[B + k] = rest[k];
    }
}

// Two codes, in the bits `mask` of x's halves, as halves (c - 8) s. Bits 0 .. 3 under 0x6400 are the half 1024 + c, bits
// 4 .. 7 under 0x5400 the half 64 + c: one logic instruction, and one multiply-add with (s, o = -1032 s or -72 s), both exact: s
// has four significant bits, and 129 and 9 times them fit a half's eleven. For keys, scales are taken 2^-4 smaller, so that
// 1032 s stays a half (and the smallest ones are still exact).
__device__ __forceinline__ uint32_t half_code(uint32_t x, uint32_t mask, uint32_t base, uint32_t s, uint32_t o) {
    uint32_t h, r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(h) : "r"(x), "r"(mask), "r"(base));     // (x & mask) | base
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(h), "r"(s), "r"(o));
    return r;
}
// The same in two steps, with off = -1032 or -72: where s changes from code to code, o would have to be fetched with it.
__device__ __forceinline__ uint32_t half_code_apart(uint32_t x, uint32_t mask, uint32_t base, uint32_t off, uint32_t s) {
    uint32_t h, r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(h) : "r"(x), "r"(mask), "r"(base));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(h), "r"(off));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(s));
    return r;
}
constexpr uint32_t CODES_LOW = 0x000F000Fu, CODES_HIGH = 0x00F000F0u;
constexpr uint32_t H2_1024 = 0x64006400u, H2_64 = 0x54005400u, H2_SMALLER = 0x2C002C00u, H2_M1032 = 0xE408E408u, H2_M72 = 0xD480D480u;
constexpr float ATT_LARGER = 16.f;       // what keys are too small by
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Whether a query saw any token, from its reference and sum: a NaN among its scores never becomes the reference.
__device__ __forceinline__ bool has_seen(float m, float sum) { return m > ATT_NONE || sum != sum; }

// Without a time of its own: the waits here are short.
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(specv::smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits, as a warp, for a phase of `bar`. Where it gives up it sets the status bit and clears `alive`, so that later waits
// end at once (the results are invalid, but every barrier is still met). A try sleeps in hardware until the phase ends or
// its time is up, so turns are few; the clock is looked at every 256 of them.
__device__ __forceinline__ void wait_phase(uint64_t* bar, uint32_t parity, bool& alive, unsigned* status) {
    uint64_t since = 0;
    for (int i = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)) && alive; ++i) {
        if (i % 256 == 0) {
            const uint64_t now = specv::global_timer_ns();
            if (since == 0) since = now;
            if (!__all_sync(0xffffffffu, now - since < ATT_WAIT_NS)) {
                atomicOr(status, SPEC_STATUS_TIMEOUT);
                alive = false;
            }
        }
    }
}

// Bits [lo, hi) of a word, the ends clamped.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
    const uint32_t below_hi = hi >= 32 ? ~0u : hi > 0 ? (1u << hi) - 1u : 0u;
    return lo >= 32 ? 0u : lo > 0 ? below_hi & (~0u << lo) : below_hi;
}
// The same value, tied to this place: keeps what is worked out from it inside its branch.
__device__ __forceinline__ uint32_t here(uint32_t v) {
    asm volatile("" : "+r"(v));
    return v;
}

// Two neighbouring bf16 or fp16 values, and back (rounded to nearest).
__device__ __forceinline__ float2 two_of(uint32_t v, int fp16) {
    if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ unsigned short one_out(float v, int fp16) {
    if (fp16) return __half_as_ushort(__float2half_rn(v));
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// What the computing warps have to know of a tile, written by the fetching warp before the tile's copies.
struct __align__(16) TileInfo {
    int pos0, pos1;          // first position of its two pages, -1 where there is none
    int b, h, r0, rows;      // sequence, key head, first row of the query block and its rows
    int len, ql;
    int flags, slot;         // where its part goes if the unit is cut
    int before_all, seen_by_all;     // a page is seen whole by every query of the block if its first position is past
                                     // the one and not past the other
};
constexpr int TILE_FIRST = 1, TILE_LAST = 2, TILE_ALONE = 4;    // of this CTA's part of the unit; the part is the unit

struct Place {
    long long start;         // of the sequence, on the line
    int b;
};

// Named barriers: computing threads and the fetching warp (keys stored; probabilities stored, with a vote), computing
// threads alone.
constexpr int BAR_KEYS = 1, BAR_PROBS = 2, BAR_COMPUTE = 3;
__device__ __forceinline__ void bar_arrive(int id, int threads) {
    asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool bar_vote(int id, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(v))
        : "memory");
    return r != 0;
}

template <int D, int WG, int NW>
__global__ void __launch_bounds__(Att<D, WG, NW>::TH, Att<D, WG, NW>::CTAS)
    attention_kernel(const __grid_constant__ AttnParams p) {
    using C = Att<D, WG, NW>;
    using BL = Block<D>;
    constexpr int TH = C::TH, CT = C::CT, NC = C::NC, NQ = C::NQ, NG = BL::NG;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(8) uint64_t s_full[C::STAGES];
    __shared__ __align__(8) uint64_t s_bar_s, s_bar_o;
    __shared__ uint32_t s_tmem, s_base[2];
    __shared__ TileInfo s_info[C::INFOS];
    __shared__ __align__(16) float s_c[NC], s_nm[NC];    // c_n, -m_n
    __shared__ __align__(16) float s_fac[NC];
    __shared__ float s_red[4][NC], s_inv[NC];
    __shared__ long long s_off[NC];                      // output row offset
    __shared__ int s_live[NC];                           // whether it is a query, not a row past q_len or none
    __shared__ long long s_scan[TH / 32 + 1];
    __shared__ Place s_place[2];

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t sm = specv::smem_addr(smem);

    if (warp == 0) tmem_alloc(&s_tmem, C::COLS);
    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) specv::mbar_init(&s_full[i], 1);
        specv::mbar_init(&s_bar_s, 1);
        specv::mbar_init(&s_bar_o, 1);
        specv::fence_mbarrier_init_cluster();
        s_base[0] = H2_1024;
        s_base[1] = H2_64;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");      // after_previous, the next kernel let in at this one's end
    // ---- the CTA's run of tiles: an equal share of the line on which each unit takes its tiles and ATT_UNIT more in front
    long long mine = 0;
    for (int b = tid; b < p.B; b += TH) mine += load_seq(p, b, blockIdx.x == 0).T + ATT_UNIT;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) s_scan[warp] = mine;
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, s_tmem, 0);
    const long long per_t = static_cast<long long>(p.Hk) * p.RB;      // units of a sequence
    long long line = 0;
    for (int w = 0; w < TH / 32; ++w) line += s_scan[w];
    line *= per_t;
    const long long A = min(static_cast<long long>(gridDim.x), line), g = blockIdx.x;     // CTAs with a share
    const long long lo = g < A ? g * line / A : line, hi = g < A ? (g + 1) * line / A : line;
    {
        // the sequences that hold places lo and hi: running sums over chunks of TH sequences
        if (tid < 2) s_place[tid].b = p.B;
        long long before = 0;
        for (int b0 = 0; b0 < p.B; b0 += TH) {
            const int b = b0 + tid;
            const long long c = b < p.B ? (load_seq(p, b, false).T + ATT_UNIT) * per_t : 0;
            long long x = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            __syncthreads();
            if (lane == 31) s_scan[warp] = x;
            __syncthreads();
            long long end = before + x;
            for (int w = 0; w < TH / 32; ++w) {
                if (w < warp) end += s_scan[w];
                before += s_scan[w];
            }
            if (c && lo < end && lo >= end - c) s_place[0] = {end - c, b};
            if (c && hi < end && hi >= end - c) s_place[1] = {end - c, b};
            if (hi < before) break;      // the same for every thread
        }
    }
    __syncthreads();
    // tiles before each place (a unit's own come after its ATT_UNIT), and the one to begin with
    Cursor at = {};
    long long from = 0, to = 0;
    for (int i = 1; i >= 0; --i) {
        const Place pl = s_place[i];
        at.b = pl.b;
        long long& n = i ? to : from;
        if (pl.b >= p.B) {
            n = line - ATT_UNIT * per_t * p.B;
        } else {
            at.s = load_seq(p, pl.b, false);
            const long long rem = (i ? hi : lo) - pl.start, len = at.s.T + ATT_UNIT;
            const int unit = static_cast<int>(rem / len);
            at.t = max(static_cast<int>(rem - unit * len) - ATT_UNIT, 0);
            at.h = unit / p.RB;
            at.rb = unit - at.h * p.RB;
            n = pl.start - ATT_UNIT * per_t * pl.b + static_cast<long long>(unit) * at.s.T + at.t;
        }
    }
    const int tiles = static_cast<int>(to - from);
    bool alive = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { wait_phase(bar, parity, alive, p.status); };

    if (warp == CT / 32) {
        // ================ the fetching warp: copies ahead, and both products of each tile
        int4 desc = make_int4(0, 0, 0, 0);
        int issued = 0, t0 = at.t;
        // the unit's query block: first row, rows, and the positions between which a page is seen whole by all of it
        int r0 = 0, rows = 0, before_all = 0, seen_by_all = 0;
        auto enter = [&] {
            r0 = at.rb * p.rpb;
            rows = min(p.rpb, p.N * p.G - r0);
            seen_by_all = at.s.len - at.s.ql + r0 / p.G - (PAGE - 1);
            before_all = p.window == 0 ? -1 : static_cast<int>(max(-1LL, static_cast<long long>(at.s.len) - at.s.ql + (r0 + rows - 1) / p.G - p.window));
            for (int n = lane; n < rows; n += 32) {        // its queries, which are read when its first tile is there
                const int r = r0 + n, i = r / p.G;
                const unsigned char* const q = static_cast<const unsigned char*>(p.q.p) +
                                               2 * (at.b * p.q.sb + i * p.q.sn + (at.h * p.G + (r - i * p.G)) * p.q.sh);
                asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
                if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 128));
            }
        };
        // lanes 0 and 1 have a page of the next tile each; their numbers are read one tile before they are needed
        int j = -1, e = -1;
        auto look = [&] {
            j = lane < 2 ? at.page_index(lane) : -1;
            e = j >= 0 ? p.table[static_cast<size_t>(at.b) * p.max_pages + j] : -1;
        };
        auto issue = [&] {
            const int st = issued % C::STAGES;
            const bool valid = e >= 0 && e < p.pages;
            if (j >= 0 && !valid) atomicOr(p.status, SPEC_STATUS_BAD_PAGE);
            const int pos = valid ? j * PAGE : -1;
            const int pos1 = __shfl_sync(0xffffffffu, pos, 1);
            const bool starts = t0 == 0, first = issued == 0 || at.t == 0, ends = at.t + 1 == at.s.T, last = ends || issued + 1 == tiles;
            if (lane == 0) {
                TileInfo& f = s_info[issued % C::INFOS];
                f.pos0 = pos, f.pos1 = pos1;
                f.b = at.b, f.h = at.h, f.r0 = r0, f.rows = rows;
                f.len = at.s.len, f.ql = at.s.ql;
                f.flags = (first ? TILE_FIRST : 0) | (last ? TILE_LAST : 0) | (starts && ends ? TILE_ALONE : 0);
                f.slot = static_cast<int>(2 * g) + (starts ? 1 : 0);
                f.before_all = before_all, f.seen_by_all = seen_by_all;
                specv::mbar_arrive_expect_tx(&s_full[st], ((pos >= 0) + (pos1 >= 0)) * BL::BYTES);
            }
            __syncwarp();
            if (valid) {
                const uint64_t policy = p.RB == 1 ? specv::policy_evict_first() : specv::policy_evict_normal();
                specv::bulk_load(smem + st * C::TILE + lane * BL::BYTES, p.pool + (static_cast<size_t>(e) * p.Hk + at.h) * BL::BYTES,
                                 BL::BYTES, &s_full[st], policy);
            }
            if (last && starts && !ends) {       // the unit's tiles end in a later CTA
                const long long end = hi + (at.s.T - at.t - 1);        // the place behind the unit's last tile: this one's is hi - 1
                desc = make_int4(at.b, at.h * p.RB + at.rb, static_cast<int>((end * A - 1) / line - g + 1), 0);
            }
            if (++issued < tiles) {
                at.next(p);
                if (at.t == 0) {
                    t0 = 0;
                    enter();
                }
                look();
            }
            __syncwarp();
        };
        if (tiles > 0) {
            enter();
            look();
            for (int i = 0; i < C::STAGES && issued < tiles; ++i) issue();
        }
        const uint32_t idesc_s = umma_idesc(NC), idesc_o = umma_idesc(C::ON) | UMMA_B_MN_MAJOR;
        const uint64_t q_desc = umma_desc(sm + C::Q, C::KQ, 128), p_desc = umma_desc(sm + C::P, C::KP, 128);
        for (int k = 0; k < tiles; ++k) {
            const bool first = s_info[k % C::INFOS].flags & TILE_FIRST;
            bar_sync(BAR_KEYS, TH);
            tmem_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) umma_ts(tbase + C::COL_S, tbase + 8 * i, q_desc + i * (2 * C::KQ >> 4), idesc_s, i > 0);
                umma_commit(&s_bar_s);
            }
            __syncwarp();
            while (bar_vote(BAR_PROBS, TH, false)) {}      // at most one turn: see the computing warps
            tmem_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < C::OK / 16; ++i)
                    umma_ts(tbase + C::COL_O, tbase + 8 * i, p_desc + i * (2 * C::KP >> 4), idesc_o, i > 0 || !first);
                umma_commit(&s_bar_o);
            }
            __syncwarp();
            if (issued < tiles) issue();       // into this tile's slot: its values were read before the vote
        }
        if (lane == 0) p.desc[g] = desc;
        // no copy is in flight into this CTA's shared memory when it is given back, even where a wait gave up
        for (int k = max(0, issued - C::STAGES); k < issued; ++k) wait(&s_full[k % C::STAGES], static_cast<uint32_t>(k / C::STAGES) & 1u);
    } else {
        // ================ the computing warps
        const int wg = warp >> 2, wq = warp & 3;
        const int tok = wq * 32 + lane;                      // this thread's lane of tensor memory
        const uint32_t tlane = tbase + (static_cast<uint32_t>(wq * 32) << 16);
        // from shared memory, so that they stay in registers: the logic instruction takes one immediate, and the compiler would
        // rather build the other constant anew each time
        const uint32_t low = *static_cast<volatile uint32_t*>(&s_base[0]), high = *static_cast<volatile uint32_t*>(&s_base[1]);
        // of the value bytes' two codes, this warp's channels have the lower or the upper one
        const bool upper = D == 128 ? wq >> 1 : wq & 1;
        const uint32_t v_mask = upper ? CODES_HIGH : CODES_LOW, v_base = upper ? high : low, v_off = upper ? H2_M72 : H2_M1032;
        const uint32_t col_o = tlane + C::COL_O + (D == 64 && wq >= 2 ? NC : 0) + wg * NW;
        unsigned long long l[NW / 2];      // this thread's part of each query's sum
#pragma unroll
        for (int n = 0; n < NW / 2; ++n) l[n] = 0ull;
        for (int k = 0; k < tiles; ++k) {
            const int st = k % C::STAGES;
            const unsigned char* const tile = smem + st * C::TILE;
            const TileInfo& f = s_info[k % C::INFOS];
            wait(&s_full[st], static_cast<uint32_t>(k / C::STAGES) & 1u);
            const int pos0 = f.pos0, pos1 = f.pos1, flags = f.flags;
            if (flags & TILE_FIRST) {
                // ---- a new unit: its queries as halves, each row scaled by a power of two into a half's range
                // (rarely run, so short: its instructions are not in the cache.) A thread takes eight channels of a row.
                constexpr int CH = D / 8, PER = (NQ * CH + CT - 1) / CT;
                uint4 raw[PER];
#pragma unroll
                for (int u = 0; u < PER; ++u) {
                    const int n = (u * CT + tid) / CH, r = f.r0 + n, i = r / p.G, hq = f.h * p.G + (r - i * p.G);
                    const bool row = n < f.rows, live = row && i < f.ql;
                    raw[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (live)
                        raw[u] = *reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.q.p) +
                                                                 2 * (f.b * p.q.sb + i * p.q.sn + hq * p.q.sh + 8 * (tid % CH)));
                    if (tid % CH == 0 && n < NQ) {
                        s_off[n] = i * p.out.sn + hq * p.out.sh;
                        s_live[n] = live;
                        s_nm[n] = -ATT_NONE;
                    }
                }
#pragma unroll
                for (int u = 0; u < PER; ++u) {
                    const int n = (u * CT + tid) / CH;
                    const float2 v[4] = {two_of(raw[u].x, p.fp16), two_of(raw[u].y, p.fp16), two_of(raw[u].z, p.fp16), two_of(raw[u].w, p.fp16)};
                    float top = 0.f;
#pragma unroll
                    for (int q = 0; q < 4; ++q) top = max3(top, fabsf(v[q].x), fabsf(v[q].y));
#pragma unroll
                    for (int o = CH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // 2^ex brings the largest magnitude to 2^10 .. 2^11 (and an infinite one nowhere)
                    const int ex = top > 0.f && top <= 3.4e38f ? 137 - max(static_cast<int>(__float_as_uint(top) >> 23), 20) : 0;
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
                    // channels in the order 0 4 1 5 2 6 3 7
                    const __half2 h[4] = {__floats2half2_rn(v[0].x * up, v[2].x * up), __floats2half2_rn(v[0].y * up, v[2].y * up),
                                          __floats2half2_rn(v[1].x * up, v[3].x * up), __floats2half2_rn(v[1].y * up, v[3].y * up)};
                    if (n < NQ) {
                        *reinterpret_cast<uint4*>(smem + C::Q + (tid % CH) * C::KQ + (n >> 3) * 128 + (n & 7) * 16) = *reinterpret_cast<const uint4*>(h);
                        if (tid % CH == 0) s_c[n] = s_live[n] ? p.scale * ATT_LARGER * __uint_as_float(static_cast<uint32_t>(127 - ex) << 23) : 0.f;
                    }
                }
                specv::fence_proxy_async_shared();
                bar_sync(BAR_COMPUTE, CT);
            }
            // ---- the scales of this warp's values: a lane has four tokens of the warp's group, pairs (0, 2) and (1, 3)
            unsigned char* const vs = smem + C::VS + warp * C::WORDS * 8;
            if (lane < C::WORDS) {
                const int q = wg * C::WORDS + lane, page = D == 128 ? q / 16 : wq >> 1, t4 = (4 * q) % PAGE, gr = wq % NG;
                const int from = page ? pos1 : pos0, left = from >= 0 ? f.len - from - t4 : 0;      // tokens that hold something
                // the tokens' scales of all groups, this one's picked out of them: a byte's place in a half is 7 up
                const unsigned char* const b = tile + page * BL::BYTES + BL::VS + t4 * NG;
                uint32_t s02, s13;
                if constexpr (D == 128) {
                    const uint4 w = *reinterpret_cast<const uint4*>(b);
                    s02 = __byte_perm(w.x, w.z, gr * 0x11 + 0x40), s13 = __byte_perm(w.y, w.w, gr * 0x11 + 0x40);
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(b);
                    s02 = __byte_perm(w.x, w.y, gr * 0x11 + 0x40), s13 = __byte_perm(w.x, w.y, gr * 0x11 + 0x62);
                }
                if (left < 4) {
                    s02 &= (left > 0 ? 0xFFu : 0u) | (left > 2 ? 0xFF00u : 0u);
                    s13 &= (left > 1 ? 0xFFu : 0u) | (left > 3 ? 0xFF00u : 0u);
                }
                s02 = (s02 & 0xFFu) << 7 | (s02 & 0xFF00u) << 15, s13 = (s13 & 0xFFu) << 7 | (s13 & 0xFF00u) << 15;
                *reinterpret_cast<uint2*>(vs + lane * 8) = make_uint2(s02, s13);
            }
            // ---- keys to halves: this thread's token, this warpgroup's groups
            {
                const int t = tok % PAGE;
                const unsigned char* const blk = tile + (tok / PAGE) * BL::BYTES;
#pragma unroll
                for (int i = 0; i < NG / WG; ++i) {
                    const int gr = wg * (NG / WG) + i;
                    const uint4 v = *reinterpret_cast<const uint4*>(blk + BL::key(gr, t));
                    const uint32_t s2 = half2_mul(blk[BL::KS + t * NG + gr] * 0x00800080u, H2_SMALLER);
                    const uint32_t ol = half2_mul(s2, H2_M1032), oh = half2_mul(s2, H2_M72);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t kr[16];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t w8 = w[q] >> 8;
                        kr[4 * q] = half_code(w[q], CODES_LOW, low, s2, ol);
                        kr[4 * q + 1] = half_code(w[q], CODES_HIGH, high, s2, oh);
                        kr[4 * q + 2] = half_code(w8, CODES_LOW, low, s2, ol);
                        kr[4 * q + 3] = half_code(w8, CODES_HIGH, high, s2, oh);
                    }
                    if (i == 0 && !(flags & TILE_FIRST)) {       // the tile before's values are read, their columns are free
                        wait(&s_bar_o, (k - 1) & 1);
                        tmem_fence_after();
                    }
                    tmem_st16(tlane + 16 * gr, kr);
                }
            }
            tmem_wait_st();
            tmem_fence_before();
            bar_arrive(BAR_KEYS, TH);
            // ---- values to halves, the first part of the tokens while the first product runs
            uint32_t vr[2 * C::WPP];
            auto values = [&](int part) {
                const int r = D == 128 ? (wq & 1) * 32 + lane : lane;
#pragma unroll
                for (int u = 0; u < C::WPP / 4; ++u) {
                    const int run = wg * (C::WORDS / 4) + part * (C::WPP / 4) + u, page = D == 128 ? run / 4 : wq >> 1;
                    const uint4 v = *reinterpret_cast<const uint4*>(tile + page * BL::BYTES + BL::value((run % 4) * 16, r));
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        const uint4 sc = *reinterpret_cast<const uint4*>(vs + (part * C::WPP + 4 * u + q) * 8);
                        vr[8 * u + 2 * q] = half_code_apart(w[q], v_mask, v_base, v_off, sc.x);
                        vr[8 * u + 2 * q + 1] = half_code_apart(w[q] >> 8, v_mask, v_base, v_off, sc.y);
                        vr[8 * u + 2 * q + 2] = half_code_apart(w[q + 1], v_mask, v_base, v_off, sc.z);
                        vr[8 * u + 2 * q + 3] = half_code_apart(w[q + 1] >> 8, v_mask, v_base, v_off, sc.w);
                    }
                }
            };
            auto put_values = [&](int part) {
#pragma unroll
                for (int i = 0; i < 2 * C::WPP / 16; ++i)
                    tmem_st16(tlane + 2 * (wg * C::WORDS + part * C::WPP) + 16 * i, vr + 16 * i);
            };
            __syncwarp();        // the warp's scales are written
            values(0);
            wait(&s_bar_s, k & 1);
            tmem_fence_after();
            put_values(0);
            if (C::VP == 2) {
                values(1);
                put_values(1);
            }
            // ---- which queries see this thread's token: all of them where the whole tile is seen by all
            const bool whole = min(pos0, pos1) > f.before_all && max(pos0, pos1) <= f.seen_by_all;
            uint32_t seen = ~0u;
            if (!whole) {
                const int from = tok < PAGE ? pos0 : pos1, at = from + tok % PAGE, base = f.len - f.ql;
                int nlo = 0, nhi = 0;
                if (from >= 0 && at < f.len) {
                    nlo = max(at - base, 0) * p.G - f.r0;
                    nhi = NC;
                    if (p.window > 0 && at >= p.sinks)
                        nhi = static_cast<int>(min(max(static_cast<long long>(at) - base + p.window, 0LL), static_cast<long long>(p.N)) * p.G) - f.r0;
                }
                seen = bit_range(nlo - wg * NW, nhi - wg * NW);      // of this thread's queries
            }
            unsigned long long x[NW / 2];
            for (bool move = flags & TILE_FIRST;; move = true) {
                uint32_t u[NW];
                tmem_load<NW>(tlane + C::COL_S + wg * NW, u);
                if (move) {
                    // the references move to ATT_BELOW under the maxima seen so far; l and, unless this is the part's first tile,
                    // O follow
                    float y[NW];
                    const uint32_t bits = here(seen);
#pragma unroll
                    for (int n = 0; n < NW; ++n) y[n] = bits >> n & 1 ? __uint_as_float(u[n]) * s_c[wg * NW + n] : -INFINITY;
                    fold_columns(y, lane, &s_red[wq][wg * NW], [](float a, float b) { return fmaxf(a, b); });
                    bar_sync(BAR_COMPUTE, CT);
                    if (tid < NQ) {
                        const float old = -s_nm[tid];
                        const float top = fmaxf(fmaxf(s_red[0][tid], s_red[1][tid]), fmaxf(s_red[2][tid], s_red[3][tid]));
                        const float now = fmaxf(top - ATT_BELOW, old);      // no token seen: -inf, and the old one stays
                        s_fac[tid] = specv::ex2(old - now);
                        s_nm[tid] = -now;
                    }
                    bar_sync(BAR_COMPUTE, CT);
#pragma unroll
                    for (int n = 0; n < NW / 2; ++n) l[n] = mul2(l[n], *reinterpret_cast<const unsigned long long*>(&s_fac[wg * NW + 2 * n]));
                    if (!(flags & TILE_FIRST)) {
#pragma unroll 1
                        for (int i = 0; i < NW; i += 8) {
                            uint32_t o[8];
                            tmem_ld(col_o + i, o);
#pragma unroll
                            for (int n = 0; n < 8; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * s_fac[wg * NW + i + n]);
                            tmem_st8(col_o + i, o);
                        }
                    }
                }
                // this token's probabilities, to shared memory as the second product's operand
                float over = -INFINITY;
                const int pt = tok % C::OK, pos = (pt & ~3) + ((pt & 1) << 1) + ((pt >> 1) & 1);       // 0 2 1 3 in each four
                unsigned char* const row = smem + C::P + (pos >> 3) * C::KP + (pos & 7) * 16 + ((D == 64 ? tok / PAGE * NC : 0) + wg * NW) / 8 * 128;
#pragma unroll
                for (int n = 0; n < NW; n += 4) {
                    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&s_c[wg * NW + n]);
                    const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(&s_nm[wg * NW + n]);
                    x[n / 2] = fma2(pack2(__uint_as_float(u[n]), __uint_as_float(u[n + 1])), c.x, m.x);
                    x[n / 2 + 1] = fma2(pack2(__uint_as_float(u[n + 2]), __uint_as_float(u[n + 3])), c.y, m.y);
                }
                if (!whole) {
                    const uint32_t bits = here(seen);
#pragma unroll
                    for (int n = 0; n < NW; n += 2) {
                        const float2 v = unpack2(x[n / 2]);
                        x[n / 2] = pack2(bits >> n & 1 ? v.x : -INFINITY, bits >> (n + 1) & 1 ? v.y : -INFINITY);
                    }
                }
#pragma unroll
                for (int n = 0; n < NW; n += 8) {
                    uint32_t h[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 v = unpack2(x[n / 2 + q]);
                        over = max3(over, v.x, v.y);
                        const float e0 = specv::ex2(v.x), e1 = specv::ex2(v.y);
                        x[n / 2 + q] = pack2(e0, e1);
                        const __half2 hv = __floats2half2_rn(e0, e1);
                        h[q] = *reinterpret_cast<const uint32_t*>(&hv);
                    }
                    *reinterpret_cast<uint4*>(row + (n / 8) * 128) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                tmem_wait_st();
                specv::fence_proxy_async_shared();
                tmem_fence_before();
                // a score that passed its reference by too much: once more, with the references moved (after which none does)
                if (!bar_vote(BAR_PROBS, TH, !move && over > ATT_SLACK)) break;
                tmem_fence_after();
            }
#pragma unroll
            for (int n = 0; n < NW / 2; ++n) l[n] = add2(l[n], x[n]);
            if (flags & TILE_LAST) {
                // ---- the part's end: O and the sums out
                wait(&s_bar_o, k & 1);
                tmem_fence_after();
                float lf[NW];
#pragma unroll
                for (int n = 0; n < NW / 2; ++n) {
                    const float2 v = unpack2(l[n]);
                    lf[2 * n] = v.x, lf[2 * n + 1] = v.y;
                    l[n] = 0ull;
                }
                fold_columns(lf, lane, &s_red[wq][wg * NW], [](float a, float b) { return a + b; });
                if (D == 64 && wq >= 2) {      // the second page's share of O, to the lanes that write
#pragma unroll 1
                    for (int i = 0; i < NW; i += 8) {
                        uint32_t o[8];
                        tmem_ld(col_o + i, o);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            *reinterpret_cast<uint32_t*>(smem + C::P + ((wg * NW + i + q) * 64 + tok - 64) * 4) = o[q];
                    }
                }
                bar_sync(BAR_COMPUTE, CT);
                const bool alone = flags & TILE_ALONE;
                if (tid < NQ) {
                    const float sum = (s_red[0][tid] + s_red[1][tid]) + (s_red[2][tid] + s_red[3][tid]), m = -s_nm[tid];
                    const bool some = s_live[tid] && has_seen(m, sum);
                    s_inv[tid] = some ? 1.f / sum : 0.f;
                    if (tid < f.rows) {
                        const int r = f.r0 + tid, i = r / p.G;
                        if (!alone) p.part_ml[static_cast<size_t>(f.slot) * p.width + tid] = make_float2(m, sum);
                        else if (p.lse)
                            p.lse[(static_cast<long long>(f.b) * p.N + i) * p.Hq + f.h * p.G + (r - i * p.G)] =
                                some ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
                    }
                }
                bar_sync(BAR_COMPUTE, CT);
                if (D == 128 || wq < 2) {
                    unsigned short* const out = static_cast<unsigned short*>(p.out.p) + f.b * p.out.sb + tok;
                    float* const part = p.part_o + (static_cast<size_t>(f.slot) * p.width + wg * NW) * D + tok;
#pragma unroll 1
                    for (int i = 0; i < NW; i += 8) {
                        uint32_t o[8];
                        tmem_ld(col_o + i, o);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const int n = wg * NW + i + q;
                            float v = __uint_as_float(o[q]);
                            if (D == 64) v += *reinterpret_cast<const float*>(smem + C::P + (n * 64 + tok) * 4);
                            if (n >= f.rows) continue;
                            // a row that sees nothing is 0 whatever its O: its columns may hold what no token's weight stands for
                            if (alone) out[s_off[n]] = one_out(s_inv[n] != 0.f ? v * s_inv[n] : 0.f, p.fp16);
                            else part[(i + q) * D] = v;
                        }
                    }
                }
                tmem_fence_before();
                bar_sync(BAR_COMPUTE, CT);      // the queries' and sums' shared memory is free again
                tmem_fence_after();
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 0) tmem_dealloc(tbase, C::COLS);
}

// Joins the parts of the unit that starts in CTA blockIdx.x of the kernel before and is cut, a warp to a query row, in
// order of the parts.
template <int D>
__global__ void __launch_bounds__(128) attention_join_kernel(const __grid_constant__ AttnParams p) {
    constexpr int E = D / 32;
    after_previous();
    const int4 u = p.desc[blockIdx.x];
    if (u.z == 0) return;
    const int lane = threadIdx.x & 31, n = blockIdx.y * 4 + (threadIdx.x >> 5);
    const int h = u.y / p.RB, r0 = (u.y - h * p.RB) * p.rpb, r = r0 + n;
    if (n >= p.rpb || r >= p.N * p.G) return;
    const int i = r / p.G, hq = h * p.G + (r - i * p.G);
    const long long g = blockIdx.x;
    auto slot = [&](int k) { return k == 0 ? 2 * g + 1 : 2 * (g + k); };
    float m = ATT_NONE;
    for (int k = lane; k < u.z; k += 32) m = fmaxf(m, p.part_ml[slot(k) * p.width + n].x);
    m = specv::warp_max(m);
    float o[E] = {}, sum = 0.f;
#pragma unroll 4
    for (int k = 0; k < u.z; ++k) {
        const float2 ml = p.part_ml[slot(k) * p.width + n];
        const float w = specv::ex2(ml.x - m);
        const float2* const part = reinterpret_cast<const float2*>(p.part_o + (slot(k) * p.width + n) * D + E * lane);
        sum = fmaf(ml.y, w, sum);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 v = part[e / 2];
            o[e] = fmaf(v.x, w, o[e]);
            o[e + 1] = fmaf(v.y, w, o[e + 1]);
        }
    }
    const int ql = p.q_len ? p.q_len[u.x] : p.N;
    const bool seen = i < ql && has_seen(m, sum);
    const float inv = 1.f / sum;
    unsigned short* const out = static_cast<unsigned short*>(p.out.p) + u.x * p.out.sb + i * p.out.sn + hq * p.out.sh + E * lane;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = one_out(seen ? o[e] * inv : 0.f, p.fp16);
    if (p.lse && lane == 0)
        p.lse[(static_cast<long long>(u.x) * p.N + i) * p.Hq + hq] = seen ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace specc
