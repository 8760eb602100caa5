/*
 * speccache.h -- C ABI of the scoring step around a verification, GB300 (sm_103a), part of libspecverify.so.
 *
 * A serving loop scores K + 1 tokens of every sequence with the target, verifies the drafts (specverify.h),
 * keeps the accepted ones and drops the rest. The calls here are the operators it needs for that, over a
 * paged key / value cache held in 4 bits:
 *  - spec_qk_norm_rope: root-mean-square norm of each query and key head and rotation by position;
 *  - spec_cache_append, spec_cache_read: keys and values quantised into their pages, and back;
 *  - spec_cache_attention: attention of the newest tokens over the cache, whole or with a sliding window and
 *    first tokens that stay visible;
 *  - spec_pages_fork, _reserve, _commit, _release, _compact: the pages' bookkeeping.
 * One round: reserve, then per layer norm_rope, append, attention; then spec_verify, then commit with its
 * accept_len.
 *
 * The cache. A pool is device memory [pages][Hk][68 D] bytes (pages_* also take [layers][pages][Hk][68 D]):
 * a page holds SPEC_CACHE_PAGE = 64 tokens, in one block of 68 D bytes per key head:
 *   [key codes 32 D][key scales 2 D][value codes 32 D][value scales 2 D].
 * Each token's 32 neighbouring channels share a scale s, held in 8 bits (5 of exponent, 3 of mantissa, no sign:
 * byte b is the half with bits b << 7; at most 896). A code c in -7..7 is held as c + 8 in 4 bits and stands
 * for c s. Quantisation: s is the representable scale nearest (even on ties) to a seventh of the group's
 * largest magnitude; c the nearest integer (even on ties) to x / s, at most 7 in magnitude, 0 where s = 0.
 * So magnitudes above 6272 saturate, and a group below 7 * 2^-18 becomes 0; NaN becomes 0. Every c s is exact in
 * bf16 and fp16.
 *   key codes   [D / 32 groups][64 tokens][16 bytes]: byte j of a token's 16 holds channel 32 g + 2 j in its low
 *               half and 32 g + 2 j + 1 in its high half;
 *   value codes [4 runs of 16 tokens][D / 2][16 tokens]: a byte holds channel r in its low half and channel
 *               r + D / 2 in its high half;
 *   scales      [64 tokens][D / 32].
 * A table is int32 [sequences][max_pages], row-major: the page that holds a sequence's tokens 64 j .. 64 j + 63,
 * or -1. refs is int32 [pages]: how many table entries name a page; 0 is free. lengths is int32 [sequences]: the
 * tokens committed.
 *
 * Conventions, those of specverify.h: device pointers of the caller's; nothing is allocated; asynchronous on
 * `stream`; every call can be captured into a CUDA graph. Arguments that the host can see are checked before
 * anything is launched (SPEC_ERR_INVALID, SPEC_ERR_UNSUPPORTED; message in spec_cache_last_error()). What is
 * on the device is checked there: a bad page or length is never followed and ORs a bit into the status word, the
 * first word of the workspace (spec_read_status, spec_clear_status). A workspace's first SPEC_CACHE_WS_HEADER
 * bytes are zeroed once before its first use and kept by the calls; 16-byte aligned; calls that share one must
 * not overlap on the GPU. Empty calls (B, N, S or the number of pairs 0) do nothing, but for a compaction without
 * sequences, which still moves the pages that are counted.
 *
 * Activations are bf16, fp16 or, for the norm and rotation, fp32 (dtype: SPEC_BF16, SPEC_FP16, SPEC_FP32), as
 * [B, N, heads, D] with any strides over B, N and heads and contiguous channels; pointers and strides (of more than
 * one entry) are multiples of 16 bytes; an output's rows must not overlap. D is 64 or 128 (the norm and rotation also 256).
 */
#ifndef SPECCACHE_H
#define SPECCACHE_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SPEC_FP16 = 2 };   /* a further value of spec_dtype's int, for the calls of this header */

#define SPEC_CACHE_PAGE 64          /* tokens of a page */
#define SPEC_CACHE_GROUP 32         /* channels that share a scale */
#define SPEC_CACHE_WS_HEADER 8192   /* bytes of a workspace that are zeroed before its first use */

/* Bits of the status word, beside specverify.h's. Of those, spec_cache_attention sets SPEC_STATUS_TIMEOUT: a wait within the
 * kernel gave up after two seconds, and the outputs are invalid. */
#define SPEC_STATUS_BAD_PAGE 4u     /* a page that was needed is missing or outside the pool */
#define SPEC_STATUS_BAD_LENGTH 8u   /* a length outside the table, or a count outside [0, N] */
#define SPEC_STATUS_NO_PAGES 16u    /* a reservation found too few free pages */
#define SPEC_STATUS_BAD_SLOT 32u    /* a sequence number outside the table, or a pair that another one excludes */

/* [B, N, heads, D] in device memory: element strides over the first three, channels contiguous. */
typedef struct {
    void* data;
    long long stride_b, stride_n, stride_h;
} spec_heads;

/* Bytes of one page's block of one key head: 68 D, or 0 for an unsupported D. */
size_t spec_cache_block_bytes(int D);

/* For each token and head: y = x / sqrt(mean(x^2) + eps) w, then the first `rotary` channels of y are rotated in
 * pairs by the angle 2 pi positions[b, n] freqs[i] / 2^64, pair i being channels (i, i + rotary / 2), or (2 i,
 * 2 i + 1) where `interleaved`. freqs: device uint64 [rotary / 2], each pair's turns a position as a fraction of
 * 2^64: the product wraps exactly, so angles of far positions keep their precision. positions: device int32
 * [B, N]. Weights: device [D] of the activations' type, or NULL for 1. rotary: a multiple of 16 up to D; 0 leaves
 * the rotation out. q and k may have different numbers of heads; either may have none (Hq or Hk 0). Outputs may
 * be the inputs; they may not overlap them otherwise. Sums and rotation in fp32, rounded once. */
spec_status spec_qk_norm_rope(const spec_heads* q, const spec_heads* k, int dtype, int B, int N, int Hq, int Hk,
                              int D, const int32_t* positions, const uint64_t* freqs, int rotary, int interleaved,
                              const void* q_weight, const void* k_weight, float eps, const spec_heads* q_out,
                              const spec_heads* k_out, void* stream);

/* Quantises k and v [B, N, Hk, D] (bf16 or fp16) into the pool: token i of sequence b goes to position start[b]
 * + i, for i < counts[b] (counts NULL: N). start, counts: device int32 [B]. A token whose page the table lacks is
 * left out (SPEC_STATUS_BAD_PAGE, or SPEC_STATUS_BAD_LENGTH where the position is outside the table). No two of
 * the call's positions may share a page's slot. Workspace: SPEC_CACHE_WS_HEADER bytes. */
spec_status spec_cache_append(void* pool, int pages, const int32_t* table, int max_pages, const int32_t* start,
                              const int32_t* counts, const spec_heads* k, const spec_heads* v, int dtype, int B,
                              int N, int Hk, int D, void* workspace, size_t workspace_bytes, void* stream);

/* The reverse: the cached values of positions start[b] + i, i < counts[b], as bf16 or fp16, exactly; other
 * outputs, and tokens whose page is missing, are 0. k_out or v_out may have a NULL data. */
spec_status spec_cache_read(const void* pool, int pages, const int32_t* table, int max_pages, const int32_t* start,
                            const int32_t* counts, const spec_heads* k_out, const spec_heads* v_out, int dtype,
                            int B, int N, int Hk, int D, void* workspace, size_t workspace_bytes, void* stream);

/* Attention of each sequence's newest tokens over its cached keys and values, their own included. Query i of
 * sequence b (i < q_len[b]; NULL: N) stands at position p = kv_len[b] - q_len[b] + i and sees the positions t <= p
 * with, where window > 0, t > p - window or t < sinks:
 *   out[b, i, h] = sum_t softmax_t(scale q[b, i, h] . key[t, h / (Hq / Hk)]) value[t, h / (Hq / Hk)].
 * A query that sees nothing (p < 0) and a row past q_len give 0, and -inf in lse, the natural logarithm of
 * the sum of exponentials (device float [B, N, Hq] or NULL). kv_len, q_len: device int32 [B]. Pages that no query
 * sees may be -1. A visible page that is missing counts as unseen (SPEC_STATUS_BAD_PAGE). Queries and outputs
 * are bf16 or fp16; Hq is a multiple of Hk; window >= 0 (0: all), sinks >= 0; N at most 1024. Scores, softmax and
 * sums in fp32; probabilities are rounded to fp16 for the product with the values, those down to 2^-21 of the largest to
 * its eleven bits and smaller ones by 2^-32 of the largest at most. The workspace size for N serves every call with up
 * to N new tokens a sequence and the same heads. */
size_t spec_cache_attention_workspace_size(int N, int Hq, int Hk, int D);
spec_status spec_cache_attention(const spec_heads* q, int dtype, const void* pool, int pages, const int32_t* table,
                                 int max_pages, const int32_t* kv_len, const int32_t* q_len, int B, int N, int Hq,
                                 int Hk, int D, float scale, int window, int sinks, const spec_heads* out,
                                 float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace for the spec_pages_* calls, spec_cache_append and spec_cache_read. */
size_t spec_pages_workspace_size(int S, int pages);

/* Sequence dst[f] becomes a copy of src[f] that shares its pages: dst's former pages are let go, src's are
 * counted once more. src, dst: device int32 [F]. A pair is left out (SPEC_STATUS_BAD_SLOT) if either number is
 * outside [0, S), or its dst is the dst of an earlier pair or the src of any. F at most 4096. */
spec_status spec_pages_fork(int32_t* table, int32_t* lengths, int32_t* refs, int S, int max_pages, int pages,
                            const int32_t* src, const int32_t* dst, int F, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Makes room for positions lengths[s] .. lengths[s] + n_new[s] - 1 that this sequence alone writes: a missing page
 * among them is taken from the free ones; a page that other sequences share is replaced, and where it holds
 * committed tokens of this one (the last, part-filled page) copied, in every layer. Pages are wanted in order of
 * (sequence, position); the k-th gets the k-th lowest free page. "Free" and "shared" are as the call finds them.
 * A sequence is served whole or not at all: not if its positions pass the table (SPEC_STATUS_BAD_LENGTH), nor if
 * the pages wanted up to and with it are more than the free ones (SPEC_STATUS_NO_PAGES). served: device int32 [S]
 * or NULL, 1 or 0. pool: [layers][pages][page_bytes], page_bytes a multiple of 16. */
spec_status spec_pages_reserve(void* pool, int layers, long long page_bytes, int32_t* table, const int32_t* lengths,
                               int32_t* refs, int S, int max_pages, int pages, const int32_t* n_new,
                               int32_t* served, void* workspace, size_t workspace_bytes, void* stream);

/* lengths[s] += advance[s] + extra, with spec_verify's accept_len as advance and extra = 1 for the token before
 * the drafts. Pages past the new length are let go (a count that reaches 0 is free), and, where window > 0, those
 * that hold no position below sinks and that no later query sees. advance: device int32 [S]. A new length
 * outside [0, 64 max_pages] is clamped (SPEC_STATUS_BAD_LENGTH); a negative advance rolls back. */
spec_status spec_pages_commit(int32_t* table, int32_t* lengths, int32_t* refs, int S, int max_pages, int pages,
                              const int32_t* advance, int extra, int window, int sinks, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Lets go of every page of the sequences slots [F] (device int32) and sets their lengths to 0. */
spec_status spec_pages_release(int32_t* table, int32_t* lengths, int32_t* refs, int S, int max_pages, int pages,
                               const int32_t* slots, int F, void* workspace, size_t workspace_bytes, void* stream);

/* Moves the pages in use to the front of the pool: with n in use, the i-th used page at or past n goes to the
 * i-th free one below n, in every layer; table and refs follow. used: device int32 [1] or NULL, n. Where a page went is
 * in the table alone: a page that is to be found again needs an entry there. */
spec_status spec_pages_compact(void* pool, int layers, long long page_bytes, int32_t* table, int32_t* refs, int S,
                               int max_pages, int pages, int32_t* used, void* workspace, size_t workspace_bytes,
                               void* stream);

/* Thread-local message describing the last non-OK status that a call of this header returned on this thread. */
const char* spec_cache_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SPECCACHE_H */
