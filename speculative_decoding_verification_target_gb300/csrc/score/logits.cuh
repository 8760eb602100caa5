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
    int stream;     // 0: the output is the input, and no mask changes it
};

// What the history, the drafts and the biases say of a token, in a word: bit 31 in the prompt, bit 30 among the drafts, bits
// 11 .. 29 the times among the output, bits 0 .. 10 the number of its bias's entry + 1.
constexpr unsigned W_PROMPT = 1u << 31, W_DRAFT = 1u << 30, W_ONE = 1u << 11, W_BIAS = W_ONE - 1, W_COUNT = W_DRAFT - W_ONE;
constexpr int LG_THREADS = 256;

// The mask's bits of the `n` <= 8 tokens from v on; `last` is its last word.
__device__ __forceinline__ unsigned mask_bits(const unsigned* mask, int v, int last, int n) {
    const int w = v >> 5, by = v & 31;
    unsigned bits = __ldg(mask + w) >> by;
    if (by + n > 32) bits |= __ldg(mask + min(w + 1, last)) << (32 - by);
    return bits & ((1u << n) - 1u);
}

// -inf where a bit is 0.
template <class T>
__device__ __forceinline__ uint4 masked(uint4 x, unsigned bits) {
    if constexpr (std::is_same_v<T, float>) {
        x.x = bits & 1u ? x.x : 0xFF800000u, x.y = bits & 2u ? x.y : 0xFF800000u;
        x.z = bits & 4u ? x.z : 0xFF800000u, x.w = bits & 8u ? x.w : 0xFF800000u;
    } else {
        auto two = [](uint32_t v, unsigned b) {
            const uint32_t keep = (b & 1u) * 0xFFFFu | (b >> 1 & 1u) * 0xFFFF0000u;
            return (v & keep) | (0xFF80FF80u & ~keep);
        };
        x.x = two(x.x, bits), x.y = two(x.y, bits >> 2), x.z = two(x.z, bits >> 4), x.w = two(x.w, bits >> 6);
    }
    return x;
}

// A CTA takes one sequence and `seg` tokens of the vocabulary, for all rows. It first copies the rows, 16 bytes at a time, with the
// mask: bandwidth bounds that. What the sequence's tokens say comes from a table in shared memory, one word a token; the few
// logits that it changes are then worked out once more, each by itself.
template <class T>
__global__ void __launch_bounds__(LG_THREADS) logits_kernel(const __grid_constant__ LogitsParams p) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    extern __shared__ unsigned s_word[];
    __shared__ unsigned s_draft[SPEC_SCORE_MAX_ROWS];
    after_previous();
    const int b = blockIdx.y, tid = threadIdx.x, last_word = (p.V - 1) / 32;
    const int v0 = blockIdx.x * p.seg, n = min(p.seg, p.V - v0);
    for (int i = tid; i < p.seg / 4; i += LG_THREADS) reinterpret_cast<uint4*>(s_word)[i] = make_uint4(0u, 0u, 0u, 0u);
    // drafts before a row: an id outside this part of the vocabulary is n or more, below 0 too
    for (int j = tid; j < p.R; j += LG_THREADS)
        s_draft[j] = p.tokens && j < p.R - 1 ? static_cast<unsigned>(p.tokens[static_cast<long long>(b) * p.T + j]) - v0 : ~0u;
    if (p.stream) {
        for (int j = 0; j < p.R; ++j) {
            const T* const in = row_of<T>(p.in, b, j) + v0;
            T* const out = row_of<T>(p.out, b, j) + v0;
            const unsigned* const mask = p.mask ? p.mask + b * p.mask_sb + j * p.mask_sr : nullptr;
            int head = 0, whole = 0;
            if (p.pieces) {
                head = min(n, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(out) & 15u)) & 15u) / static_cast<int>(sizeof(T)));
                whole = (n - head) / E;
            }
            const uint4* const from = reinterpret_cast<const uint4*>(in + head);
            uint4* const to = reinterpret_cast<uint4*>(out + head);
#pragma unroll 4
            for (int i = tid; i < whole; i += LG_THREADS) {
                uint4 x = from[i];
                if (mask) x = masked<T>(x, mask_bits(mask, v0 + head + i * E, last_word, E));
                to[i] = x;
            }
            for (int i = tid; i < n - whole * E; i += LG_THREADS) {      // the rest, one by one
                const int at = i < head ? i : i + whole * E;
                out[at] = !mask || mask_bits(mask, v0 + at, last_word, 1) ? in[at] : from_float<T>(-INFINITY);
            }
        }
    }
    __syncthreads();
    if (p.bias_tokens) {
        for (int i = tid; i < p.biases; i += LG_THREADS) {
            const unsigned v = static_cast<unsigned>(p.bias_tokens[static_cast<long long>(b) * p.biases + i]) - v0;
            if (v < static_cast<unsigned>(n)) atomicMax(&s_word[v], static_cast<unsigned>(i + 1));
        }
        __syncthreads();
    }
    if (p.history) {
        const int len = min(max(p.lengths[b], 0), p.L), pr = p.prompt ? p.prompt[b] : 0;
        const int* const h = p.history + static_cast<long long>(b) * p.L;
#pragma unroll 4
        for (int i = tid; i < len; i += LG_THREADS) {
            const unsigned v = static_cast<unsigned>(__ldg(h + i)) - v0;
            if (v >= static_cast<unsigned>(n)) continue;
            if (i < pr) atomicOr(&s_word[v], W_PROMPT);
            else atomicAdd(&s_word[v], W_ONE);
        }
    }
    for (int j = tid; j < p.R; j += LG_THREADS)
        if (s_draft[j] < static_cast<unsigned>(n)) atomicOr(&s_word[s_draft[j]], W_DRAFT);
    __syncthreads();
    const float rep = p.repetition ? p.repetition[b] : 1.f, freq = p.frequency ? p.frequency[b] : 0.f,
                pres = p.presence ? p.presence[b] : 0.f;
    for (int v = tid; v < n; v += LG_THREADS) {
        const unsigned w = s_word[v];
        if (!w) continue;
        const float add = w & W_BIAS ? p.bias[static_cast<long long>(b) * p.biases + (w & W_BIAS) - 1] : 0.f;
        unsigned count = (w & W_COUNT) / W_ONE;
#pragma unroll 4
        for (int j = 0; j < p.R; ++j) {
            if (j && s_draft[j - 1] == static_cast<unsigned>(v)) ++count;
            if (!(w & (W_PROMPT | W_BIAS)) && !count) continue;
            if (p.mask && !mask_bits(p.mask + b * p.mask_sb + j * p.mask_sr, v0 + v, last_word, 1)) continue;
            float y = to_float(row_of<T>(p.in, b, j)[v0 + v]) + add;
            if (count || w & W_PROMPT) y = y > 0.f ? y / rep : y * rep;
            if (count) y = y - freq * static_cast<float>(count) - pres;
            row_of<T>(p.out, b, j)[v0 + v] = from_float<T>(y);
        }
    }
}

}  // namespace specs
