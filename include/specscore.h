/*
 * specscore.h -- C ABI of the operators between the target's last layer and a verification, GB300 (sm_103a), part of
 * libspecverify.so.
 *
 * What a serving loop runs on the tokens that it is about to verify, one behind the other:
 *  - spec_residual_norm: the residual's addition and the root-mean-square norm, to the activations' type or to
 *    8-bit integers with a scale per token;
 *  - spec_quantize_rows: 8-bit integers with a scale per token, without a norm (an attention's output, inner values of a
 *    feed-forward part, and weights once: a row is then an output channel);
 *  - spec_int8_matmul: the product of 8-bit integers with scales for each token and each output channel, the
 *    vocabulary's among others;
 *  - spec_process_logits: biases, penalties for repeated tokens and grammar masks on the logits, for every row
 *    of a draft chain with the drafts before it.
 * Then spec_verify (specverify.h) on the processed target and draft logits.
 *
 * Conventions, those of specverify.h and speccache.h: device pointers of the caller's; nothing is allocated; asynchronous
 * on `stream`; every call can be captured into a CUDA graph. Arguments that the host can see are checked before anything
 * is launched (SPEC_ERR_INVALID, SPEC_ERR_UNSUPPORTED; message in spec_score_last_error()). Empty calls (no tokens, no
 * rows, no channels) do nothing. No call needs its data aligned beyond its type; rows that all begin on 16 bytes are faster.
 * B <= 65535, N <= 1048576 (R below), B N <= 4194304, C <= 1048576.
 * Outputs may not overlap the inputs, but for those that are named as possibly the same. An output's rows must not overlap.
 */
#ifndef SPECSCORE_H
#define SPECSCORE_H

#include "speccache.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SPEC_INT8 = 3 };   /* a further value of the type arguments of this header */

#define SPEC_SCORE_MAX_D 32768          /* values of a row of spec_residual_norm and spec_quantize_rows */
#define SPEC_SCORE_MAX_K 131071         /* products of a sum: the longest that 32 bits always hold */
#define SPEC_SCORE_MAX_ROWS 65          /* logits rows of a sequence */
#define SPEC_SCORE_MAX_HISTORY 500000   /* tokens of a history */
#define SPEC_SCORE_MAX_BIASES 1024      /* biases of a sequence */
#define SPEC_SCORE_WS_HEADER 256        /* bytes of a workspace that are zeroed before its first use */

/* Rows [B, N] of values in device memory: element strides over both, values contiguous. */
typedef struct {
    void* data;
    long long stride_b, stride_n;
} spec_rows;

/* For each token: r = x + residual, rounded to the activations' type (residual NULL: r = x), and
 *   v = r w / sqrt(mean(r^2) + eps),   w: device [D] of the activations' type, or NULL for 1.
 * residual_out receives r (NULL without a residual). out receives v rounded once to the activations' type (out_type =
 * dtype), or in 8 bits (out_type = SPEC_INT8): with p = r w rounded to fp32 (exact for bf16 and fp16) and m the
 * row's largest |p|, each code is the integer nearest to 127 p / m, even on ties, decided exactly; 0 where m = 0. scale
 * (device float [B, N]) receives m / 127 / sqrt(mean(r^2) + eps): v is about code times scale. A row with an infinity or a NaN
 * in p gets codes 0 and the scale NaN. Sums in fp32: a row whose squares' sum passes 3.4e38 counts as infinitely long, and squares below
 * 1e-38 lose digits or all (which matters where eps is as small).
 * dtype: SPEC_BF16, SPEC_FP16 or SPEC_FP32. residual_out may be x or residual, out (not in 8 bits) may be x or
 * residual; not both the same. 1 <= D <= SPEC_SCORE_MAX_D. */
spec_status spec_residual_norm(const spec_rows* x, const spec_rows* residual, int dtype, int B, int N, int D,
                               const void* weight, float eps, const spec_rows* residual_out, const spec_rows* out,
                               int out_type, float* scale, void* stream);

/* The same codes without norm and weight: code = the integer nearest to 127 x / m, scale = m / 127. */
spec_status spec_quantize_rows(const spec_rows* x, int dtype, int B, int N, int D, const spec_rows* out, float* scale,
                               void* stream);

/* out[b, n, c] = (sum_k a[b, n, k] w[c, k]) a_scale[b, n] w_scale[c] + bias[c], a and w 8-bit integers in -128..127.
 * The sum is exact (integers of 32 bits); it, the scales' product, the product of both and, with a bias, its sum with that are
 * rounded to fp32 each, and the result to out_type (SPEC_BF16, SPEC_FP16, SPEC_FP32). a: rows [B, N] of K; w: rows [C] of
 * K, w_stride apart; scales and bias (or NULL) device float, contiguous. 1 <= K <= SPEC_SCORE_MAX_K. The workspace, 16-byte aligned,
 * has its first SPEC_SCORE_WS_HEADER bytes zeroed once before its first use; its first word is the status word (SPEC_STATUS_TIMEOUT: a
 * wait within the kernel gave up after two seconds and the outputs are invalid). The size for T tokens, C channels and K serves
 * every call with up to T tokens, C channels and K products. Calls that share a workspace must not overlap on the GPU. */
size_t spec_int8_matmul_workspace_size(int tokens, int C, int K);
spec_status spec_int8_matmul(const spec_rows* a, const float* a_scale, const void* w, long long w_stride,
                             const float* w_scale, const float* bias, int B, int N, int C, int K, const spec_rows* out,
                             int out_type, void* workspace, size_t workspace_bytes, void* stream);

/* Logits [B, R, V] (bf16 or fp32) of R tokens of each sequence, as they are sampled from. Row j of sequence b comes after its
 * history[b, 0 .. lengths[b]), of which the first prompt[b] tokens are the prompt and the others output, and after the drafts
 * tokens[b, 0 .. j), which count as output. With n the times that a token is among the output, y = x + bias, then
 *   y = y > 0 ? y / repetition[b] : y repetition[b]     where the token is in the prompt or the output,
 *   y = y - frequency[b] n - (n > 0 ? presence[b] : 0),
 *   y = -inf                                            where bit (token % 32) of mask[b, j, token / 32] is 0,
 * in fp32, rounded once; the quotient of bf16 logits is y times the rounded 1 / repetition[b]. Each part is left out where its
 * pointer is NULL. history: device int32 [B, L] with lengths [B] and prompt [B] (NULL: all output); a length is taken as at least 0
 * and at most L. tokens: device int32 [B, T], T >= R - 1. Tokens outside [0, V) are passed over, so -1 pads. bias_tokens: device int32
 * [B, biases], bias: device float of the same shape; of entries with the same token the last counts. repetition (> 0), frequency,
 * presence: device float [B]. mask: device 32-bit words, the rows' ceil(V / 32) contiguous, with any strides (0: one mask for several
 * rows); bits past V are not looked at. A row whose mask allows nothing is -inf throughout: no row to verify. out may be logits.
 * R <= SPEC_SCORE_MAX_ROWS, V <= 262144. */
spec_status spec_process_logits(const spec_rows* logits, int dtype, int B, int R, int V, const int32_t* tokens, int T,
                                const int32_t* history, const int32_t* lengths, const int32_t* prompt, int L,
                                const float* repetition, const float* frequency, const float* presence,
                                const int32_t* bias_tokens, const float* bias, int biases, const uint32_t* mask,
                                long long mask_stride_b, long long mask_stride_r, const spec_rows* out, void* stream);

/* Thread-local message describing the last non-OK status that a call of this header returned on this thread. */
const char* spec_score_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SPECSCORE_H */
