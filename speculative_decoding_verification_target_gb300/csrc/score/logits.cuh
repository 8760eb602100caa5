// Biases, penalties for repeated tokens and grammar masks on the logits of a draft chain.
#pragma once
#include "rows.cuh"

namespace specs {

struct LogitsParams {
    Rows in, out;
    const int *tokens, *history, *lengths, *prompt, *bias_tokens;
    const float *repetition, *frequency, *presence, *bias;
    const unsigned* mask;
    long long mask_sb, mask_sr;
    int R, V, T, L, biases;
    int seg;        // tokens of the vocabulary that a CTA takes
    int pieces;     // every row and its output begin alike within 16 bytes
    int together;   // every row of a sequence begins alike within 16 bytes
    int stream;     // 0: the output is the input, and no mask changes it
};

// What the history, the drafts and the biases say of a token, in a word: bit 31 in the prompt, bit 30 among the drafts, bits
// 11 .. 29 the times among the output, bits 0 .. 10 the number of its bias's entry + 1.
constexpr unsigned W_PROMPT = 1u << 31, W_DRAFT = 1u << 30, W_ONE = 1u << 11, W_BIAS = W_ONE - 1, W_COUNT = W_DRAFT - W_ONE;
constexpr int LG_SEG = 8192, LG_THREADS = 256, LG_CTAS = 4;      // at most; CTAs of an SM
// Once all is counted, a word is the number that is taken off the logit: 0 for a token that nothing is said of, -0 where nothing is
// taken off but the repetition counts. Tokens with a bias or among the drafts are kept in a list, and their words are 0.
constexpr int LG_LIST = SPEC_SCORE_MAX_BIASES + SPEC_SCORE_MAX_ROWS;

// The mask's bits of the `n` <= 8 tokens from v on; `last` is its last word.
__device__ __forceinline__ unsigned mask_bits(const unsigned* mask, int v, int last, int n) {
    const int w = v >> 5, by = v & 31;
    unsigned bits = __ldg(mask + w) >> by;
    if (by + n > 32) bits |= __ldg(mask + min(w + 1, last)) << (32 - by);
    return bits & ((1u << n) - 1u);
}

// -inf where a bit is 0. For 16-bit values `keep` holds the words' bits to be kept for each of the 256 bytes of a mask: an entry is a
// read of 16 bytes where working it out takes as many instructions.
template <class T>
__device__ __forceinline__ uint4 masked(uint4 x, unsigned bits, const uint4* keep) {
    if constexpr (std::is_same_v<T, float>) {
        x.x = bits & 1u ? x.x : 0xFF800000u, x.y = bits & 2u ? x.y : 0xFF800000u;
        x.z = bits & 4u ? x.z : 0xFF800000u, x.w = bits & 8u ? x.w : 0xFF800000u;
    } else {
        const uint4 k = keep[bits];
        auto two = [](uint32_t v, uint32_t m) { return (v & m) | (0xFF80FF80u & ~m); };
        x.x = two(x.x, k.x), x.y = two(x.y, k.y), x.z = two(x.z, k.z), x.w = two(x.w, k.w);
    }
    return x;
}
__device__ __forceinline__ uint4 kept_bits(unsigned bits) {
    // four bits to the bytes of a word, each byte to 0 or 255, and twice for a half
    const uint32_t lo = ((bits & 15u) * 0x00204081u & 0x01010101u) * 255u, hi = ((bits >> 4) * 0x00204081u & 0x01010101u) * 255u;
    return make_uint4(__byte_perm(lo, 0, 0x1100), __byte_perm(lo, 0, 0x3322), __byte_perm(hi, 0, 0x1100), __byte_perm(hi, 0, 0x3322));
}

// `n` <= 8 bits of the table's flags from v on; a word behind the last is there.
__device__ __forceinline__ unsigned flag_bits(const unsigned* flags, int v, int n) {
    const unsigned low = flags[v >> 5] >> (v & 31);
    return ((v & 31) + n > 32 ? low | flags[(v >> 5) + 1] << (32 - (v & 31)) : low) & ((1u << n) - 1u);
}

// Where token v's word stands. 16-bit logits take eight words a piece: the first and the second four of them in parts of their own,
// so that neighbouring lanes read neighbouring 16 bytes.
template <int E>
__device__ __forceinline__ int word_at(int v, int seg) {
    return E == 4 ? v : ((v >> 3) + (v >> 2 & 1) * (seg / 8 + 1)) * 4 + (v & 3);
}

// The words of tokens v .. v + E - 1, v - from a multiple of four, `from` the same for every lane.
template <int E>
__device__ __forceinline__ void words_of(const unsigned* s_word, int v, int from, int seg, uint32_t (&w)[E]) {
    if (from == 0) {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const uint4 q = *reinterpret_cast<const uint4*>(s_word + word_at<E>(v + i, seg));
            w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
        }
        return;
    }
    uint32_t t[E + 4];
#pragma unroll
    for (int i = 0; i < E + 4; i += 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(s_word + word_at<E>(v - from + i, seg));
        t[i] = q.x, t[i + 1] = q.y, t[i + 2] = q.z, t[i + 3] = q.w;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] = from == 1 ? t[i + 1] : from == 2 ? t[i + 2] : t[i + 3];
}

// A CTA takes one sequence and `seg` tokens of the vocabulary, for all rows. What the sequence's tokens say comes first, from a
// pass over its history, into a table in shared memory: a word for each token, and a bit for each that is not 0. Then the rows
// go by, 16 bytes of a row at a time, and all rows at a place one behind the other, since the table says the same to them: bandwidth
// bounds that. A piece without a bit is copied, with the mask; in the others every value goes through the one formula, which leaves
// those that nothing is said of as they are. Listed tokens come last, each by itself. 128 sequences of 21 rows of 151936 in bf16 with
// histories of up to 32768 tokens take 292 us, 84% of the copy rate; 64 of 6 rows of 128256 with masks and biases 61.8 us (49%), where
// the table, made once for six rows, and the masks count for more.
template <class T, bool MASK>
__global__ void __launch_bounds__(LG_THREADS, LG_CTAS) logits_kernel(const __grid_constant__ LogitsParams p) {
    constexpr int E = 16 / static_cast<int>(sizeof(T)), U = MASK ? 3 : 6;
    extern __shared__ unsigned s_word[];                     // [seg + 8], then the bits [seg / 32 + 1]
    __shared__ unsigned s_draft[SPEC_SCORE_MAX_ROWS], s_list[LG_LIST], s_listed;
    __shared__ unsigned short s_token[LG_LIST];
    __shared__ uint4 s_keep[MASK && E == 8 ? 256 : 1];
    after_previous();
    const int b = blockIdx.y, tid = threadIdx.x, threads = blockDim.x, last_word = (p.V - 1) / 32;
    const int v0 = blockIdx.x * p.seg, n = min(p.seg, p.V - v0);
    unsigned* const s_flag = s_word + p.seg + 8;
    if (tid == 0) s_listed = 0u;
    if (MASK && E == 8)
        for (int i = tid; i < 256; i += threads) s_keep[i] = kept_bits(i);
    auto at = [&](int v) { return word_at<E>(v, p.seg); };
    for (int i = tid; i < p.seg / 4 + 2; i += threads) reinterpret_cast<uint4*>(s_word)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i <= p.seg / 32; i += threads) s_flag[i] = 0u;
    // drafts before a row: an id outside this part of the vocabulary is n or more, below 0 too
    for (int j = tid; j < p.R; j += threads)
        s_draft[j] = p.tokens && j < p.R - 1 ? static_cast<unsigned>(p.tokens[static_cast<long long>(b) * p.T + j]) - v0 : ~0u;
    __syncthreads();
    auto mark = [&](unsigned v) { atomicOr(&s_flag[v / 32], 1u << (v % 32)); };
    if (p.bias_tokens) {
        for (int i = tid; i < p.biases; i += threads) {
            const unsigned v = static_cast<unsigned>(p.bias_tokens[static_cast<long long>(b) * p.biases + i]) - v0;
            if (v < static_cast<unsigned>(n)) atomicMax(&s_word[at(v)], static_cast<unsigned>(i + 1)), mark(v);
        }
        __syncthreads();
    }
    if (p.history) {
        const int len = min(max(p.lengths[b], 0), p.L), pr = p.prompt ? p.prompt[b] : 0;
        const int* const h = p.history + static_cast<long long>(b) * p.L;
        auto count = [&](int id, int i) {
            const unsigned v = static_cast<unsigned>(id) - v0;
            if (v >= static_cast<unsigned>(n)) return;
            unsigned* const word = &s_word[at(v)];
            if (i < pr) atomicOr(word, W_PROMPT);
            else atomicAdd(word, W_ONE);
            mark(v);
        };
        const int fours = (reinterpret_cast<uintptr_t>(h) & 15u) == 0 ? len / 4 : 0;
#pragma unroll 2
        for (int i = tid; i < fours; i += threads) {
            const int4 t = __ldg(reinterpret_cast<const int4*>(h) + i);
            count(t.x, 4 * i), count(t.y, 4 * i + 1), count(t.z, 4 * i + 2), count(t.w, 4 * i + 3);
        }
#pragma unroll 4
        for (int i = 4 * fours + tid; i < len; i += threads) count(__ldg(h + i), i);
    }
    for (int j = tid; j < p.R; j += threads)
        if (s_draft[j] < static_cast<unsigned>(n)) atomicOr(&s_word[at(s_draft[j])], W_DRAFT), mark(s_draft[j]);
    __syncthreads();
    const float rep = p.repetition ? p.repetition[b] : 1.f, freq = p.frequency ? p.frequency[b] : 0.f,
                pres = p.presence ? p.presence[b] : 0.f, per_rep = 1.f / rep;
    // the word of a token of the text, n times among the output; n as a float without a conversion
    auto said = [&](unsigned n) {
        const unsigned off = n ? __float_as_uint(fmaf(freq, __uint_as_float(n | 0x4B000000u) - 8388608.f, pres)) : 0u;
        return off ? off : 0x80000000u;
    };
    for (int i = tid; i < p.seg / 4; i += threads)
        for (unsigned rest = s_flag[i / 8] >> 4 * (i % 8) & 15u; rest; rest &= rest - 1) {
            const int v = 4 * i + __ffs(rest) - 1;
            unsigned& word = s_word[at(v)];
            const unsigned w = word;
            if (w & (W_BIAS | W_DRAFT)) {
                const unsigned to = atomicAdd(&s_listed, 1u);
                s_list[to] = w;
                s_token[to] = static_cast<unsigned short>(v);
                word = 0u;
            } else {
                word = said((w & W_COUNT) / W_ONE);
            }
        }
    __syncthreads();
    // A quotient by a divisor known in advance (Brisebarre, Muller and Raina, IEEE Transactions on Computers 53, 2004): x times the
    // rounded reciprocal and times what that lacks, joined by one rounding. Repetitions near either end of fp32's range, whose
    // reciprocals are not whole, divide, value by value. Before bf16's rounding the reciprocal alone does: its half step of fp32 is a
    // 2^16th of the half step behind it, the second product costs 5% to 9% of a call, and a division for the ends 2% to 4%.
    const float rest = fmaf(-rep, per_rep, 1.f) * per_rep;
    const bool known = E == 8 || (rep >= 5.4210109e-20f && rep <= 1.8446744e19f);      // 2^-64, 2^64
    auto simple = [&](float x, unsigned w) {
        const float off = __uint_as_float(w);
        if constexpr (E == 8) {
            return fmaf(x, w ? (x > 0.f ? per_rep : rep) : 1.f, -off);
        } else {
            const bool up = w && __float_as_uint(x) - 1u < 0x7F7FFFFFu;      // 0 < x < infinity
            return fmaf(x, up ? per_rep : w ? rep : 1.f, up ? fmaf(x, rest, -off) : -off);
        }
    };
    auto one = [&](float x, unsigned w) { return known || !w || !(x > 0.f) ? simple(x, w) : x / rep - __uint_as_float(w); };
    const int together = p.together ? p.R : 1;
    for (int first = 0; first < p.R; first += together) {
        const int past = min(first + together, p.R);
        const T* const in = row_of<T>(p.in, b, first) + v0;
        T* const out = row_of<T>(p.out, b, first) + v0;
        const unsigned* const mask = MASK ? p.mask + b * p.mask_sb + first * p.mask_sr : nullptr;
        int head = 0, whole = 0;
        if (p.pieces && known) {
            head = min(n, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(out) & 15u)) & 15u) / static_cast<int>(sizeof(T)));
            whole = (n - head) / E;
        }
        const bool even = E == 8 && head % 8 == 0;           // a piece's bits are a byte of the mask
        for (int i = tid; i < whole; i += threads) {
            const int v = head + i * E;
            const unsigned flags = flag_bits(s_flag, v, E);
            if (!p.stream && !flags) continue;
            uint32_t w[E];                                   // what the table says, once for all rows
            if (flags) words_of<E>(s_word, v, v & 3, p.seg, w);
            const T* from = in + v;
            T* to = out + v;
            const unsigned* bits_from = mask;
            for (int j = first; j < past; j += U) {      // the loads of U rows are on their way together
                uint4 x[U];
                unsigned bits[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    if (j + k >= past) break;
                    x[k] = *reinterpret_cast<const uint4*>(from + k * p.in.sn);
                    if (MASK) bits[k] = even ? __ldg(reinterpret_cast<const unsigned char*>(bits_from + k * p.mask_sr) + (v0 + v) / 8) : mask_bits(bits_from + k * p.mask_sr, v0 + v, last_word, E);
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    if (j + k >= past) break;
                    if (flags) {
                        uint4 y = x[k];
                        if constexpr (E == 4) {
                            y.x = __float_as_uint(simple(__uint_as_float(y.x), w[0])), y.y = __float_as_uint(simple(__uint_as_float(y.y), w[1]));
                            y.z = __float_as_uint(simple(__uint_as_float(y.z), w[2])), y.w = __float_as_uint(simple(__uint_as_float(y.w), w[3]));
                        } else {
                            auto two = [&](uint32_t u, uint32_t a, uint32_t c) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(simple(__uint_as_float(u << 16), a),
                                                                               simple(__uint_as_float(u & 0xFFFF0000u), c));
                                return *reinterpret_cast<const uint32_t*>(&h);
                            };
                            y = make_uint4(two(y.x, w[0], w[1]), two(y.y, w[2], w[3]), two(y.z, w[4], w[5]), two(y.w, w[6], w[7]));
                        }
                        x[k] = y;
                    }
                    *reinterpret_cast<uint4*>(to + k * p.out.sn) = MASK ? masked<T>(x[k], bits[k], s_keep) : x[k];
                }
                from += U * p.in.sn;
                to += U * p.out.sn;
                bits_from += MASK ? U * p.mask_sr : 0;
            }
        }
        for (int j = first; j < past; ++j)
            for (int i = tid; i < n - whole * E; i += threads) {      // the rest, one by one
                const int v = i < head ? i : i + whole * E;
                const unsigned w = s_word[at(v)];
                T* const to = row_of<T>(p.out, b, j) + v0 + v;
                const T x = row_of<T>(p.in, b, j)[v0 + v];
                if (MASK && !mask_bits(p.mask + b * p.mask_sb + j * p.mask_sr, v0 + v, last_word, 1)) *to = from_float<T>(-INFINITY);
                else if (w) *to = from_float<T>(one(to_float(x), w));
                else if (p.stream) *to = x;
            }
    }
    __syncthreads();      // the rows are written: listed tokens' logits as they were
    const int listed = static_cast<int>(s_listed);
    for (int i = tid; i < listed * p.R; i += threads) {
        const int j = i / listed, v = s_token[i - j * listed];
        const unsigned w = s_list[i - j * listed];
        if (MASK && !mask_bits(p.mask + b * p.mask_sb + j * p.mask_sr, v0 + v, last_word, 1)) continue;
        float x = to_float(row_of<T>(p.in, b, j)[v0 + v]);
        unsigned count = (w & W_COUNT) / W_ONE;
        if (w & W_DRAFT)
            for (int k = 0; k < j; ++k) count += s_draft[k] == static_cast<unsigned>(v);
        if (w & W_BIAS) x += p.bias[static_cast<long long>(b) * p.biases + (w & W_BIAS) - 1];
        if (!count && !(w & (W_PROMPT | W_BIAS))) continue;
        if (count || w & W_PROMPT) x = one(x, said(count));
        row_of<T>(p.out, b, j)[v0 + v] = from_float<T>(x);
    }
}

}  // namespace specs
