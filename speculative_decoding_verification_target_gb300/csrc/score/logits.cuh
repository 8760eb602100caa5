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
};

// A CTA takes one sequence and SEG tokens of the vocabulary, for all rows. What the history, the drafts and the biases say of
// those tokens stands in a word each: bit 31 in the prompt, bits 11 .. 30 the times among the output, bits 0 .. 10 the
// number of its bias's entry + 1.
constexpr int SEG = 8192;
constexpr unsigned W_PROMPT = 1u << 31, W_ONE = 1u << 11, W_BIAS = W_ONE - 1;

template <class T>
__global__ void __launch_bounds__(256) logits_kernel(const __grid_constant__ LogitsParams p) {
    __shared__ unsigned s_word[SEG];
    after_previous();
    const int b = blockIdx.y;
    const unsigned v0 = blockIdx.x * SEG, n = min(static_cast<unsigned>(SEG), p.V - v0);   // an id below 0 is a large one
    for (unsigned i = threadIdx.x; i < n; i += 256) s_word[i] = 0u;
    __syncthreads();
    if (p.bias_tokens)
        for (int i = threadIdx.x; i < p.biases; i += 256) {
            const unsigned v = static_cast<unsigned>(p.bias_tokens[static_cast<long long>(b) * p.biases + i]) - v0;
            if (v < n) atomicMax(&s_word[v], static_cast<unsigned>(i + 1));
        }
    __syncthreads();
    if (p.history) {
        const int len = min(max(p.lengths[b], 0), p.L), pr = p.prompt ? p.prompt[b] : 0;
        for (int i = threadIdx.x; i < len; i += 256) {
            const unsigned v = static_cast<unsigned>(p.history[static_cast<long long>(b) * p.L + i]) - v0;
            if (v >= n) continue;
            if (i < pr) atomicOr(&s_word[v], W_PROMPT);
            else atomicAdd(&s_word[v], W_ONE);
        }
    }
    const float rep = p.repetition ? p.repetition[b] : 1.f, freq = p.frequency ? p.frequency[b] : 0.f,
                pres = p.presence ? p.presence[b] : 0.f;
    for (int j = 0; j < p.R; ++j) {
        __syncthreads();
        if (j && p.tokens && threadIdx.x == 0) {
            const unsigned v = static_cast<unsigned>(p.tokens[static_cast<long long>(b) * p.T + j - 1]) - v0;
            if (v < n) s_word[v] += W_ONE;
        }
        __syncthreads();
        const T* const in = row_of<T>(p.in, b, j) + v0;
        T* const out = row_of<T>(p.out, b, j) + v0;
        const unsigned* const mask = p.mask ? p.mask + b * p.mask_sb + j * p.mask_sr + v0 / 32 : nullptr;
        for (unsigned i = threadIdx.x; i < n; i += 256) {
            const T x = in[i];
            const unsigned w = s_word[i];
            if (mask && !(mask[i / 32] >> (i % 32) & 1u)) out[i] = from_float<T>(-INFINITY);
            else if (!w) out[i] = x;
            else {
                float y = to_float(x);
                if (w & W_BIAS) y += p.bias[static_cast<long long>(b) * p.biases + (w & W_BIAS) - 1];
                const unsigned count = (w & ~W_PROMPT) / W_ONE;
                if (w >= W_ONE) y = y > 0.f ? y / rep : y * rep;
                if (count) y = y - freq * static_cast<float>(count) - pres;
                out[i] = from_float<T>(y);
            }
        }
    }
}

}  // namespace specs
