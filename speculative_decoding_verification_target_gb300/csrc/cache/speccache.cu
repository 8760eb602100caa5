// Host side of the C ABI declared in include/speccache.h: argument checks and launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "speccache.h"
#include "append.cuh"
#include "attention.cuh"
#include "norm_rope.cuh"
#include "pages.cuh"

namespace specc {
namespace {

thread_local char g_err[512] = "";

spec_status fail(spec_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return s;
}

spec_status launched(const char* what, cudaError_t e) {
    return e == cudaSuccess ? SPEC_OK : fail(SPEC_ERR_CUDA, "%s failed: %s", what, cudaGetErrorString(e));
}

constexpr int MAX_B = 65535, MAX_TOKENS = 1 << 20, MAX_HEADS = 1024, MAX_Q = 1024, MAX_PAIRS = 4096;

size_t elem_bytes(int dtype) { return dtype == SPEC_FP32 ? 4 : 2; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A [B, N, heads, D] argument: present, and every row 16-byte aligned (the stride of a single entry says nothing).
spec_status check_heads(const spec_heads* t, const char* name, int dtype, int B, int N, int heads) {
    if (!t || !t->data) return fail(SPEC_ERR_INVALID, "%s must not be NULL", name);
    const long long per = 16 / static_cast<long long>(elem_bytes(dtype));
    if (!aligned16(t->data) || (B > 1 && t->stride_b % per) || (N > 1 && t->stride_n % per) || (heads > 1 && t->stride_h % per))
        return fail(SPEC_ERR_INVALID, "%s: the pointer and every stride must be a multiple of 16 bytes", name);
    return SPEC_OK;
}

// An output: its rows must not share elements, as those of a stride below D do.
spec_status check_out(const spec_heads* t, const char* name, int dtype, int B, int N, int heads, int D) {
    const spec_status s = check_heads(t, name, dtype, B, N, heads);
    if (s != SPEC_OK) return s;
    auto apart = [&](int n, long long stride) { return n <= 1 || stride >= D || stride <= -D; };
    if (!apart(B, t->stride_b) || !apart(N, t->stride_n) || !apart(heads, t->stride_h))
        return fail(SPEC_ERR_INVALID, "%s: rows overlap: strides must be at least D = %d", name, D);
    return SPEC_OK;
}

spec_status check_sizes(int B, int N, int heads, int max_n) {
    if (B < 0 || B > MAX_B) return fail(SPEC_ERR_INVALID, "B must be in [0, %d], got %d", MAX_B, B);
    if (N < 0 || N > max_n) return fail(SPEC_ERR_INVALID, "N must be in [0, %d], got %d", max_n, N);
    if (heads < 1 || heads > MAX_HEADS) return fail(SPEC_ERR_INVALID, "heads must be in [1, %d], got %d", MAX_HEADS, heads);
    return SPEC_OK;
}

spec_status check_workspace(const void* ws, size_t bytes, size_t need) {
    if (!ws || !aligned16(ws)) return fail(SPEC_ERR_INVALID, "workspace must be 16-byte aligned device memory");
    if (bytes < need) return fail(SPEC_ERR_INVALID, "workspace has %zu bytes, %zu needed", bytes, need);
    return SPEC_OK;
}

spec_status check_cache_dim(int D) {
    return D == 64 || D == 128 ? SPEC_OK : fail(SPEC_ERR_UNSUPPORTED, "D must be 64 or 128, got %d", D);
}

spec_status check_half_type(int dtype) {
    return dtype == SPEC_BF16 || dtype == SPEC_FP16 ? SPEC_OK
                                                    : fail(SPEC_ERR_UNSUPPORTED, "dtype must be bf16 or fp16, got %d", dtype);
}

spec_status check_table(const void* pool, int pages, const void* table, int max_pages) {
    if (!pool || !aligned16(pool)) return fail(SPEC_ERR_INVALID, "pool must be 16-byte aligned device memory");
    if (!table) return fail(SPEC_ERR_INVALID, "table must not be NULL");
    if (pages < 1 || max_pages < 1) return fail(SPEC_ERR_INVALID, "pages and max_pages must be at least 1");
    if (static_cast<long long>(max_pages) * PAGE > 2147483647LL)
        return fail(SPEC_ERR_INVALID, "max_pages is limited to %d", 2147483647 / PAGE);
    return SPEC_OK;
}

Heads heads_of(const spec_heads* t) { return {t->data, t->stride_b, t->stride_n, t->stride_h}; }

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

#define SPECC_TRY(expr)                        \
    do {                                       \
        const spec_status try_s = (expr);      \
        if (try_s != SPEC_OK) return try_s;    \
    } while (0)

// A launch whose CTAs may take their places while the kernel before still runs; each waits for that kernel's end by itself.
template <class P>
cudaError_t launch_behind(void (*fn)(const P), const P& p, dim3 grid, int threads, cudaStream_t st, size_t smem = 0) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

// ------------------------------------------------------------------------------------- norm and rotation
template <class T>
auto norm_rope_as(int head, bool interleaved, bool whole) -> void (*)(const NormParams) {
    static constexpr void (*fns[3][2][2])(const NormParams) = {
        {{norm_rope_kernel<T, 64, false, false>, norm_rope_kernel<T, 64, false, true>},
         {norm_rope_kernel<T, 64, true, false>, norm_rope_kernel<T, 64, true, true>}},
        {{norm_rope_kernel<T, 128, false, false>, norm_rope_kernel<T, 128, false, true>},
         {norm_rope_kernel<T, 128, true, false>, norm_rope_kernel<T, 128, true, true>}},
        {{norm_rope_kernel<T, 256, false, false>, norm_rope_kernel<T, 256, false, true>},
         {norm_rope_kernel<T, 256, true, false>, norm_rope_kernel<T, 256, true, true>}}};
    return fns[head][interleaved ? 1 : 0][whole ? 1 : 0];
}

// ------------------------------------------------------------------------------------------------ tokens
spec_status check_tokens(const void* pool, int pages, const int32_t* table, int max_pages, const int32_t* start, int dtype,
                         int B, int N, int Hk, int D, void* ws, size_t ws_bytes) {
    SPECC_TRY(check_half_type(dtype));
    SPECC_TRY(check_cache_dim(D));
    SPECC_TRY(check_sizes(B, N, Hk, MAX_TOKENS));
    if (B == 0 || N == 0) return SPEC_OK;
    SPECC_TRY(check_table(pool, pages, table, max_pages));
    if (!start) return fail(SPEC_ERR_INVALID, "start must not be NULL");
    return check_workspace(ws, ws_bytes, SPEC_CACHE_WS_HEADER);
}

TokensParams tokens_params(const void* pool, int pages, const int32_t* table, int max_pages, const int32_t* start,
                           const int32_t* counts, const spec_heads* k, const spec_heads* v, int B, int N, int Hk, void* ws) {
    TokensParams p = {};
    p.pool = static_cast<unsigned char*>(const_cast<void*>(pool));
    p.table = table;
    p.start = start;
    p.counts = counts;
    if (k) p.k = heads_of(k);
    if (v) p.v = heads_of(v);
    p.pages = pages;
    p.max_pages = max_pages;
    p.B = B;
    p.N = N;
    p.Hk = Hk;
    p.status = static_cast<unsigned*>(ws);
    return p;
}

// --------------------------------------------------------------------------------------------- attention
// The queries that read a key head, in equal blocks of at most 64 rows, each in the narrowest kernel that holds it: a block
// costs the conversion of its tiles once, so one wide block is cheaper than two narrow ones (four sequences of 100001 to 131072
// tokens, 8 key heads of 128: 64 rows 266 us as one block, 304 us as two of 32; 48 rows 203 and 284 us as two of 24; 40 rows 203
// and 284 us). The kernel of 49 to 64 rows spills, 232 bytes of stores and 268 of loads at heads of 128: nine warps leave a thread
// 96 registers. 80 rows in one block, as two warpgroups of 40 columns, spilled 660 bytes under that limit and were as slow as two
// blocks (438 and 433 us at the time), which says nothing of one pass with registers to hold it.
struct AttSplit {
    int blocks, rows, wg, nw;
};
AttSplit att_split(int rows) {
    const int blocks = (rows + 63) / 64, per = (rows + blocks - 1) / blocks;
    const int wg = per > 32 ? 2 : 1;
    return {blocks, per, wg, wg == 1 ? (per + 7) / 8 * 8 : per <= 48 ? 24 : 32};
}

// Workspace: header, the cut units' descriptions, and two parts for each CTA that there can be.
struct AttLayout {
    size_t desc, ml, o, total;
};
AttLayout att_layout(const AttSplit& s, int D) {
    const size_t ctas = ATT_MAX_CTAS / s.wg, width = s.wg * s.nw;
    AttLayout w;
    w.desc = SPEC_CACHE_WS_HEADER;
    w.ml = w.desc + ctas * sizeof(int4);
    w.o = w.ml + 2 * ctas * width * sizeof(float2);
    w.total = w.o + 2 * ctas * width * D * sizeof(float);
    return w;
}

template <int D, int WG, int NW>
spec_status attend_as(const AttnParams& p, cudaStream_t st) {
    using C = Att<D, WG, NW>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(SPEC_ERR_CUDA, "device query failed");
    static std::atomic<unsigned> ready{0};       // devices whose limit of dynamic shared memory is raised
    const unsigned bit = dev < 32 ? 1u << dev : 0u;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(attention_kernel<D, WG, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return fail(SPEC_ERR_CUDA, "attention kernel attribute failed: %s", cudaGetErrorString(e));
        ready.fetch_or(bit, std::memory_order_release);
    }
    const int sms = sm_count();
    if (sms < 1) return fail(SPEC_ERR_CUDA, "device query failed");
    const long long tiles = static_cast<long long>(p.B) * p.Hk * p.RB * ((p.max_pages + 1) / 2);     // at most
    const int ctas = static_cast<int>(std::min<long long>({static_cast<long long>(C::CTAS) * sms, ATT_MAX_CTAS / WG, tiles}));
    SPECC_TRY(launched("attention", launch_behind(attention_kernel<D, WG, NW>, p, dim3(ctas), C::TH, st, C::SMEM)));
    return launched("attention's join", launch_behind(attention_join_kernel<D>, p, dim3(ctas, (p.rpb + 3) / 4), 128, st));
}

template <int D>
spec_status attend(const AttnParams& p, const AttSplit& s, cudaStream_t st) {
    if (s.wg == 1) {
        if (s.nw == 8) return attend_as<D, 1, 8>(p, st);
        if (s.nw == 16) return attend_as<D, 1, 16>(p, st);
        if (s.nw == 24) return attend_as<D, 1, 24>(p, st);
        return attend_as<D, 1, 32>(p, st);
    }
    if (s.nw == 24) return attend_as<D, 2, 24>(p, st);
    return attend_as<D, 2, 32>(p, st);
}

// ------------------------------------------------------------------------------------------------- pages
size_t pages_scratch_ints(int S, int pages) { return 3 * static_cast<size_t>(S) + 3 * static_cast<size_t>(pages) + 16; }

// EMPTY: a call on no sequences has something to do, on the counts alone.
template <bool EMPTY = false>
spec_status check_pages(const void* table, const void* refs, int S, int max_pages, int pages, void* ws, size_t ws_bytes,
                        size_t need) {
    if (S < 0 || S > (1 << 20)) return fail(SPEC_ERR_INVALID, "S must be in [0, %d], got %d", 1 << 20, S);
    if (S == 0 && !EMPTY) return SPEC_OK;
    if ((S > 0 && !table) || !refs) return fail(SPEC_ERR_INVALID, "table and refs must not be NULL");
    if (pages < 1 || max_pages < 1) return fail(SPEC_ERR_INVALID, "pages and max_pages must be at least 1");
    if (static_cast<long long>(max_pages) * PAGE > 2147483647LL)
        return fail(SPEC_ERR_INVALID, "max_pages is limited to %d", 2147483647 / PAGE);
    return check_workspace(ws, ws_bytes, need);
}

spec_status check_pool(const void* pool, int layers, long long page_bytes) {
    if (!pool || !aligned16(pool)) return fail(SPEC_ERR_INVALID, "pool must be 16-byte aligned device memory");
    if (layers < 1 || page_bytes < 16 || page_bytes % 16)
        return fail(SPEC_ERR_INVALID, "layers must be at least 1 and page_bytes a positive multiple of 16");
    return SPEC_OK;
}

PagesParams pages_params(int32_t* table, int32_t* lengths, int32_t* refs, int S, int max_pages, int pages, void* ws) {
    PagesParams p = {};
    p.table = table;
    p.lengths = lengths;
    p.refs = refs;
    p.S = S;
    p.M = max_pages;
    p.P = pages;
    p.status = static_cast<unsigned*>(ws);
    p.scratch = reinterpret_cast<int*>(static_cast<unsigned char*>(ws) + SPEC_CACHE_WS_HEADER);
    return p;
}

// The bookkeeping kernels run as one cluster: two CTAs up to 8192 pages, where barriers cost more than the walk over the
// counts, else eight. A reservation for 64 sequences that need no page, and a compaction without moves, in us:
//   pages          512          4096         8192         12288        16384        32768        65536        262144
//   two CTAs       8.2   6.8    8.8   6.9    8.7   8.2    9.4   9.4    11.1  11.8   19.7  22.8   52.9  64.6   194   231
//   four           8.5   6.9    9.1   6.9    8.7   7.6    9.3   7.7    9.9   8.1    13.6  12.4   24.3  23.2   122   120
//   eight          9.8   7.6    10.3  7.6    9.7   8.0    10.3  7.8    10.6  7.7    11.2  9.0    14.9  13.1   67    66
cudaError_t launch_cluster(void (*fn)(const PagesParams), const PagesParams& p, int ctas, cudaStream_t st) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(PG_THREADS);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, p);
}
int cluster_for(int pages) { return pages <= 8192 ? 2 : PG_CLUSTER; }

}  // namespace
}  // namespace specc

using namespace specc;

extern "C" {

const char* spec_cache_last_error(void) { return g_err; }

size_t spec_cache_block_bytes(int D) { return D == 64 || D == 128 ? static_cast<size_t>(68) * D : 0; }

spec_status spec_qk_norm_rope(const spec_heads* q, const spec_heads* k, int dtype, int B, int N, int Hq, int Hk, int D,
                              const int32_t* positions, const uint64_t* freqs, int rotary, int interleaved,
                              const void* q_weight, const void* k_weight, float eps, const spec_heads* q_out,
                              const spec_heads* k_out, void* stream) {
    if (dtype != SPEC_BF16 && dtype != SPEC_FP16 && dtype != SPEC_FP32)
        return fail(SPEC_ERR_UNSUPPORTED, "dtype must be bf16, fp16 or fp32, got %d", dtype);
    if (D != 64 && D != 128 && D != 256) return fail(SPEC_ERR_UNSUPPORTED, "D must be 64, 128 or 256, got %d", D);
    if (Hq < 0 || Hk < 0) return fail(SPEC_ERR_INVALID, "Hq and Hk must not be negative");
    SPECC_TRY(check_sizes(B, N, Hq + Hk, MAX_TOKENS));
    if (rotary < 0 || rotary > D || rotary % 16) return fail(SPEC_ERR_INVALID, "rotary must be a multiple of 16 in [0, D], got %d", rotary);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(SPEC_ERR_INVALID, "eps must be finite and not negative");
    if (B == 0 || N == 0) return SPEC_OK;
    if (Hq > 0) {
        SPECC_TRY(check_heads(q, "q", dtype, B, N, Hq));
        SPECC_TRY(check_out(q_out, "q_out", dtype, B, N, Hq, D));
    }
    if (Hk > 0) {
        SPECC_TRY(check_heads(k, "k", dtype, B, N, Hk));
        SPECC_TRY(check_out(k_out, "k_out", dtype, B, N, Hk, D));
    }
    if (rotary && (!positions || !freqs)) return fail(SPEC_ERR_INVALID, "positions and freqs must not be NULL");
    if (!aligned16(q_weight) || !aligned16(k_weight)) return fail(SPEC_ERR_INVALID, "weights must be 16-byte aligned");
    const int sms = sm_count();
    if (sms < 1) return fail(SPEC_ERR_CUDA, "device query failed");
    NormParams p = {};
    if (Hq > 0) p.q = heads_of(q), p.qo = heads_of(q_out);
    if (Hk > 0) p.k = heads_of(k), p.ko = heads_of(k_out);
    p.positions = positions;
    p.freqs = reinterpret_cast<const unsigned long long*>(freqs);
    p.qw = q_weight;
    p.kw = k_weight;
    p.tokens = static_cast<long long>(B) * N;
    p.N = N;
    p.Hq = Hq;
    p.Hk = Hk;
    p.rotary = rotary;
    p.eps = eps;
    // few tokens: a token's heads are split over warps until the card has 32 warps an SM
    const int rpw = 256 / D;
    p.parts = static_cast<int>(std::max<long long>(1, std::min<long long>((Hq + Hk + rpw - 1) / rpw, 32LL * sms / p.tokens)));
    const long long units = p.tokens * p.parts, ctas = (units + NORM_WARPS - 1) / NORM_WARPS;
    if (ctas > 2147483647LL) return fail(SPEC_ERR_INVALID, "too many tokens: B N is limited to 2^31");
    const int head = D == 64 ? 0 : D == 128 ? 1 : 2;
    const bool whole = rotary == D;
    void (*const fn)(const NormParams) = dtype == SPEC_BF16   ? norm_rope_as<__nv_bfloat16>(head, interleaved, whole)
                                         : dtype == SPEC_FP16 ? norm_rope_as<__half>(head, interleaved, whole)
                                                              : norm_rope_as<float>(head, interleaved, whole);
    return launched("norm and rotation", launch_behind(fn, p, dim3(static_cast<unsigned>(ctas)), NORM_WARPS * 32, static_cast<cudaStream_t>(stream)));
}

spec_status spec_cache_append(void* pool, int pages, const int32_t* table, int max_pages, const int32_t* start,
                              const int32_t* counts, const spec_heads* k, const spec_heads* v, int dtype, int B, int N, int Hk,
                              int D, void* workspace, size_t workspace_bytes, void* stream) {
    SPECC_TRY(check_tokens(pool, pages, table, max_pages, start, dtype, B, N, Hk, D, workspace, workspace_bytes));
    if (B == 0 || N == 0) return SPEC_OK;
    SPECC_TRY(check_heads(k, "k", dtype, B, N, Hk));
    SPECC_TRY(check_heads(v, "v", dtype, B, N, Hk));
    const TokensParams p = tokens_params(pool, pages, table, max_pages, start, counts, k, v, B, N, Hk, workspace);
    const dim3 grid(2 * Hk, (N + PAGE - 2) / PAGE + 1, B);   // a run of N tokens touches at most that many pages
    void (*const fn)(const TokensParams) = dtype == SPEC_BF16 ? (D == 64 ? append_kernel<__nv_bfloat16, 64> : append_kernel<__nv_bfloat16, 128>)
                                                             : (D == 64 ? append_kernel<__half, 64> : append_kernel<__half, 128>);
    return launched("append", launch_behind(fn, p, grid, TOK_THREADS, static_cast<cudaStream_t>(stream)));
}

spec_status spec_cache_read(const void* pool, int pages, const int32_t* table, int max_pages, const int32_t* start,
                            const int32_t* counts, const spec_heads* k_out, const spec_heads* v_out, int dtype, int B, int N,
                            int Hk, int D, void* workspace, size_t workspace_bytes, void* stream) {
    SPECC_TRY(check_tokens(pool, pages, table, max_pages, start, dtype, B, N, Hk, D, workspace, workspace_bytes));
    if (B == 0 || N == 0) return SPEC_OK;
    const bool has_k = k_out && k_out->data, has_v = v_out && v_out->data;
    if (has_k) SPECC_TRY(check_out(k_out, "k_out", dtype, B, N, Hk, D));
    if (has_v) SPECC_TRY(check_out(v_out, "v_out", dtype, B, N, Hk, D));
    if (!has_k && !has_v) return fail(SPEC_ERR_INVALID, "k_out and v_out must not both be NULL");
    const TokensParams p = tokens_params(pool, pages, table, max_pages, start, counts, has_k ? k_out : nullptr,
                                         has_v ? v_out : nullptr, B, N, Hk, workspace);
    const dim3 grid(2 * Hk, (N + PAGE - 2) / PAGE + 1, B);
    void (*const fn)(const TokensParams) = dtype == SPEC_BF16 ? (D == 64 ? read_kernel<__nv_bfloat16, 64> : read_kernel<__nv_bfloat16, 128>)
                                                             : (D == 64 ? read_kernel<__half, 64> : read_kernel<__half, 128>);
    return launched("read", launch_behind(fn, p, grid, TOK_THREADS, static_cast<cudaStream_t>(stream)));
}

size_t spec_cache_attention_workspace_size(int N, int Hq, int Hk, int D) {
    if (N < 1 || N > MAX_Q || Hk < 1 || Hq < Hk || Hq > MAX_HEADS || Hq % Hk || (D != 64 && D != 128)) return 0;
    size_t most = 0;      // fewer queries can take a wider kernel: 64 rows are one block of 64, 65 are two of 33 in 48 columns
    for (int n = 1; n <= N; ++n) most = std::max(most, att_layout(att_split(n * (Hq / Hk)), D).total);
    return most;
}

spec_status spec_cache_attention(const spec_heads* q, int dtype, const void* pool, int pages, const int32_t* table,
                                 int max_pages, const int32_t* kv_len, const int32_t* q_len, int B, int N, int Hq, int Hk,
                                 int D, float scale, int window, int sinks, const spec_heads* out, float* lse,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    SPECC_TRY(check_half_type(dtype));
    SPECC_TRY(check_cache_dim(D));
    SPECC_TRY(check_sizes(B, N, Hq, MAX_Q));
    if (Hk < 1 || Hq % Hk) return fail(SPEC_ERR_INVALID, "Hq must be a multiple of Hk, got %d and %d", Hq, Hk);
    if (!std::isfinite(scale)) return fail(SPEC_ERR_INVALID, "scale must be finite");
    if (window < 0 || sinks < 0) return fail(SPEC_ERR_INVALID, "window and sinks must not be negative");
    if (B == 0 || N == 0) return SPEC_OK;
    SPECC_TRY(check_heads(q, "q", dtype, B, N, Hq));
    SPECC_TRY(check_out(out, "out", dtype, B, N, Hq, D));
    SPECC_TRY(check_table(pool, pages, table, max_pages));
    if (!kv_len) return fail(SPEC_ERR_INVALID, "kv_len must not be NULL");
    const AttSplit split = att_split(N * (Hq / Hk));
    const AttLayout w = att_layout(split, D);
    SPECC_TRY(check_workspace(workspace, workspace_bytes, w.total));
    AttnParams p = {};
    p.q = heads_of(q);
    p.out = heads_of(out);
    p.pool = static_cast<const unsigned char*>(pool);
    p.table = table;
    p.kv_len = kv_len;
    p.q_len = q_len;
    p.lse = lse;
    p.status = static_cast<unsigned*>(workspace);
    p.pages = pages;
    p.max_pages = max_pages;
    p.B = B;
    p.N = N;
    p.Hq = Hq;
    p.Hk = Hk;
    p.window = window;
    p.sinks = sinks;
    p.scale = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    p.G = Hq / Hk;
    p.RB = split.blocks;
    p.rpb = split.rows;
    p.width = split.wg * split.nw;
    p.fp16 = dtype == SPEC_FP16;
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    p.desc = reinterpret_cast<int4*>(ws + w.desc);
    p.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    p.part_o = reinterpret_cast<float*>(ws + w.o);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return D == 64 ? attend<64>(p, split, st) : attend<128>(p, split, st);
}

size_t spec_pages_workspace_size(int S, int pages) {
    if (S < 0 || pages < 0) return 0;
    return SPEC_CACHE_WS_HEADER + (pages_scratch_ints(S, pages) * sizeof(int) + 15) / 16 * 16;
}

spec_status spec_pages_fork(int32_t* table, int32_t* lengths, int32_t* refs, int S, int max_pages, int pages,
                            const int32_t* src, const int32_t* dst, int F, void* workspace, size_t workspace_bytes,
                            void* stream) {
    if (F < 0 || F > MAX_PAIRS) return fail(SPEC_ERR_INVALID, "F must be in [0, %d], got %d", MAX_PAIRS, F);
    SPECC_TRY(check_pages(table, refs, S, max_pages, pages, workspace, workspace_bytes, SPEC_CACHE_WS_HEADER));
    if (F == 0 || S == 0) return SPEC_OK;
    if (!lengths || !src || !dst) return fail(SPEC_ERR_INVALID, "lengths, src and dst must not be NULL");
    PagesParams p = pages_params(table, lengths, refs, S, max_pages, pages, workspace);
    p.a = src;
    p.b = dst;
    p.n = F;
    return launched("fork", launch_behind(fork_kernel, p, dim3(F), 256, static_cast<cudaStream_t>(stream)));
}

spec_status spec_pages_reserve(void* pool, int layers, long long page_bytes, int32_t* table, const int32_t* lengths,
                               int32_t* refs, int S, int max_pages, int pages, const int32_t* n_new, int32_t* served,
                               void* workspace, size_t workspace_bytes, void* stream) {
    SPECC_TRY(check_pages(table, refs, S, max_pages, pages, workspace, workspace_bytes, spec_pages_workspace_size(S, pages)));
    if (S == 0) return SPEC_OK;
    SPECC_TRY(check_pool(pool, layers, page_bytes));
    if (!lengths || !n_new) return fail(SPEC_ERR_INVALID, "lengths and n_new must not be NULL");
    const int sms = sm_count();
    if (sms < 1) return fail(SPEC_ERR_CUDA, "device query failed");
    PagesParams p = pages_params(table, const_cast<int32_t*>(lengths), refs, S, max_pages, pages, workspace);
    p.pool = static_cast<unsigned char*>(pool);
    p.layers = layers;
    p.page_bytes = page_bytes;
    p.a = n_new;
    p.out = served;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    SPECC_TRY(launched("reserve", launch_cluster(reserve_kernel, p, cluster_for(pages), st)));
    return launched("reserve's copies", launch_behind(reserve_copy_kernel, p, dim3(2 * sms), COPY_THREADS, st));
}

spec_status spec_pages_commit(int32_t* table, int32_t* lengths, int32_t* refs, int S, int max_pages, int pages,
                              const int32_t* advance, int extra, int window, int sinks, void* workspace,
                              size_t workspace_bytes, void* stream) {
    SPECC_TRY(check_pages(table, refs, S, max_pages, pages, workspace, workspace_bytes, SPEC_CACHE_WS_HEADER));
    if (window < 0 || sinks < 0) return fail(SPEC_ERR_INVALID, "window and sinks must not be negative");
    if (S == 0) return SPEC_OK;
    if (!lengths || !advance) return fail(SPEC_ERR_INVALID, "lengths and advance must not be NULL");
    PagesParams p = pages_params(table, lengths, refs, S, max_pages, pages, workspace);
    p.a = advance;
    p.extra = extra;
    p.window = window;
    p.sinks = sinks;
    return launched("commit", launch_behind(commit_kernel, p, dim3(S), 128, static_cast<cudaStream_t>(stream)));
}

spec_status spec_pages_release(int32_t* table, int32_t* lengths, int32_t* refs, int S, int max_pages, int pages,
                               const int32_t* slots, int F, void* workspace, size_t workspace_bytes, void* stream) {
    if (F < 0 || F > (1 << 20)) return fail(SPEC_ERR_INVALID, "F must be in [0, %d], got %d", 1 << 20, F);
    SPECC_TRY(check_pages(table, refs, S, max_pages, pages, workspace, workspace_bytes, SPEC_CACHE_WS_HEADER));
    if (F == 0 || S == 0) return SPEC_OK;
    if (!lengths || !slots) return fail(SPEC_ERR_INVALID, "lengths and slots must not be NULL");
    PagesParams p = pages_params(table, lengths, refs, S, max_pages, pages, workspace);
    p.a = slots;
    p.n = F;
    return launched("release", launch_behind(release_kernel, p, dim3(F), 128, static_cast<cudaStream_t>(stream)));
}

spec_status spec_pages_compact(void* pool, int layers, long long page_bytes, int32_t* table, int32_t* refs, int S,
                               int max_pages, int pages, int32_t* used, void* workspace, size_t workspace_bytes,
                               void* stream) {
    SPECC_TRY(check_pages<true>(table, refs, S, max_pages, pages, workspace, workspace_bytes, spec_pages_workspace_size(S, pages)));
    SPECC_TRY(check_pool(pool, layers, page_bytes));
    const int sms = sm_count();
    if (sms < 1) return fail(SPEC_ERR_CUDA, "device query failed");
    PagesParams p = pages_params(table, nullptr, refs, S, max_pages, pages, workspace);
    p.pool = static_cast<unsigned char*>(pool);
    p.layers = layers;
    p.page_bytes = page_bytes;
    p.out = used;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    SPECC_TRY(launched("compact's plan", launch_cluster(compact_plan_kernel, p, cluster_for(pages), st)));
    return launched("compact's moves", launch_behind(compact_move_kernel, p, dim3(16 * sms), COPY_THREADS, st));
}

}  // extern "C"
