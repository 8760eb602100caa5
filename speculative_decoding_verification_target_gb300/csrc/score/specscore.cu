// Host side of the C ABI declared in include/specscore.h: argument checks and launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "specscore.h"
#include "logits.cuh"
#include "matmul.cuh"
#include "norm.cuh"
#include "norm_threads.h"
#include "product.cuh"

namespace specs {
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

#define SPECS_TRY(expr)                        \
    do {                                       \
        const spec_status try_s = (expr);      \
        if (try_s != SPEC_OK) return try_s;    \
    } while (0)

constexpr int MAX_B = 65535, MAX_N = 1 << 20, MAX_V = 262144, MAX_C = 1 << 20;
constexpr long long MAX_TOKENS = 1 << 22;      // B N

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

spec_status check_tokens(int B, int N) {
    if (B < 0 || B > MAX_B) return fail(SPEC_ERR_INVALID, "B must be in [0, %d], got %d", MAX_B, B);
    if (N < 0 || N > MAX_N) return fail(SPEC_ERR_INVALID, "N must be in [0, %d], got %d", MAX_N, N);
    if (static_cast<long long>(B) * N > MAX_TOKENS)
        return fail(SPEC_ERR_INVALID, "B N must be at most %lld, got %lld", MAX_TOKENS, static_cast<long long>(B) * N);
    return SPEC_OK;
}

// Rows [B, N] of values of `bytes` each: present, and the pointer on a value of its type.
spec_status check_rows(const spec_rows* t, const char* name, size_t bytes) {
    if (!t || !t->data) return fail(SPEC_ERR_INVALID, "%s must not be NULL", name);
    if (reinterpret_cast<uintptr_t>(t->data) % bytes) return fail(SPEC_ERR_INVALID, "%s: the pointer must be a multiple of %zu bytes", name, bytes);
    return SPEC_OK;
}

// Arrays of 32-bit words, or NULL.
struct Words {
    const void* p;
    const char* name;
};
spec_status check_words(std::initializer_list<Words> all) {
    for (const Words& w : all)
        if (reinterpret_cast<uintptr_t>(w.p) % 4) return fail(SPEC_ERR_INVALID, "%s: the pointer must be a multiple of 4 bytes", w.name);
    return SPEC_OK;
}

// An output: two of its rows must not share elements. Rows of one index lie `width` or more apart; where both have several, one
// index's steps must pass the whole reach of the other.
spec_status check_out(const spec_rows* t, const char* name, size_t bytes, int B, int N, long long width) {
    SPECS_TRY(check_rows(t, name, bytes));
    const long long sb = B > 1 ? std::llabs(t->stride_b) : 0, sn = N > 1 ? std::llabs(t->stride_n) : 0;
    const bool ok = (B <= 1 || sb >= width) && (N <= 1 || sn >= width) &&
                    (B <= 1 || N <= 1 || sb >= sn * (N - 1) + width || sn >= sb * (B - 1) + width);
    return ok ? SPEC_OK : fail(SPEC_ERR_INVALID, "%s: rows overlap: strides must keep rows of %lld values apart", name, width);
}

// An output in an input's place: row for row.
spec_status check_same(const spec_rows* out, const char* name, const spec_rows* x, const spec_rows* y, int B, int N) {
    for (const spec_rows* in : {x, y})
        if (in && in->data == out->data && ((B > 1 && in->stride_b != out->stride_b) || (N > 1 && in->stride_n != out->stride_n)))
            return fail(SPEC_ERR_INVALID, "%s in an input's place must have its strides", name);
    return SPEC_OK;
}

size_t type_bytes(int dtype) { return dtype == SPEC_INT8 ? 1 : dtype == SPEC_FP32 ? 4 : 2; }

spec_status check_type(int dtype) {
    return dtype == SPEC_BF16 || dtype == SPEC_FP16 || dtype == SPEC_FP32
               ? SPEC_OK
               : fail(SPEC_ERR_UNSUPPORTED, "dtype must be bf16, fp16 or fp32, got %d", dtype);
}

Rows rows_of(const spec_rows* t) { return t ? Rows{t->data, t->stride_b, t->stride_n} : Rows{nullptr, 0, 0}; }

// A launch whose CTAs may take their places while the kernel before still runs; each waits for that kernel's end by itself.
template <class P>
cudaError_t launch_behind(void (*fn)(const P), const P& p, dim3 grid, int threads, cudaStream_t st, size_t smem = 0, int cluster = 1) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

// ---------------------------------------------------------------------------------------- norm and codes
// Rows that begin and end on 16 bytes throughout, and codes on as many values. Of the others, 16-bit rows that begin alike take what
// pieces they hold (norm_peel_kernel), the rest go value by value.
bool whole_pieces(const NormParams& p, size_t e, bool codes, int B) {
    const int per = 16 / static_cast<int>(e);
    auto fits = [&](const Rows& t, size_t bytes) {
        return !t.p || (reinterpret_cast<uintptr_t>(t.p) % bytes == 0 && (B <= 1 || t.sb % per == 0) && (p.N <= 1 || t.sn % per == 0));
    };
    return p.D % per == 0 && fits(p.x, 16) && fits(p.res, 16) && fits(p.res_out, 16) && fits(p.out, codes ? per : 16) && aligned16(p.weight);
}

// Rows that begin alike within 16 bytes, one token's of x, residual and 16-bit outputs.
bool alike_rows(const NormParams& p, size_t e, bool codes, int B) {
    auto as_x = [&](const Rows& t) {
        return !t.p || ((reinterpret_cast<uintptr_t>(t.p) - reinterpret_cast<uintptr_t>(p.x.p)) % 16 == 0 &&
                        (B <= 1 || (t.sb - p.x.sb) * static_cast<long long>(e) % 16 == 0) && (p.N <= 1 || (t.sn - p.x.sn) * static_cast<long long>(e) % 16 == 0));
    };
    return as_x(p.res) && as_x(p.res_out) && (codes || as_x(p.out));
}

template <class T, bool CODES, bool VEC, bool FULL>
auto norm_of(int slots) -> void (*)(const NormParams) {
    if constexpr (VEC) return slots == 1 ? norm_rows_kernel<T, CODES, 1, VEC, FULL> : slots == 2 ? norm_rows_kernel<T, CODES, 2, VEC, FULL>
                                                                                          : norm_rows_kernel<T, CODES, 4, VEC, FULL>;
    else return slots <= 4 ? norm_rows_kernel<T, CODES, 4, VEC, FULL> : norm_rows_kernel<T, CODES, 16, VEC, FULL>;
}

template <class T, bool CODES>
spec_status norm_as(NormParams p, bool vec, bool peel, int sms, cudaStream_t st) {
    if constexpr (sizeof(T) == 2) {
        if (peel && p.D >= 256 && p.D <= 16384) {
            const int slots = p.D > 4096 || p.rows > 4LL * sms ? 4 : 2;
            p.tpr = ((p.D / 8 + slots - 1) / slots + 31) / 32 * 32;
            const int per = std::max(1, 128 / p.tpr), threads = per * p.tpr;
            const long long ctas = std::min((p.rows + per - 1) / per, static_cast<long long>(sms) * std::max(1, 512 / threads));
            const size_t smem = p.weight ? ((static_cast<size_t>(p.D) + 7) / 8 * 8 + 8) * 2 : 0;
            return launched("norm", launch_behind(slots == 4 ? norm_peel_kernel<T, CODES, 4> : norm_peel_kernel<T, CODES, 2>, p,
                                                  dim3(static_cast<unsigned>(ctas)), threads, st, smem));
        }
    }
    const int pieces = vec ? p.D / (16 / static_cast<int>(sizeof(T))) : p.D, most = vec ? 4 : 16;
    if (pieces > 512 * most)
        return launched("norm", launch_behind(norm_long_kernel<T, CODES>, p, dim3(static_cast<unsigned>(p.rows)), 512, st));
    const bool full = p.norm || p.weight || p.res.p;
    const NormThreads t = norm_threads(p.rows, pieces, vec, CODES, full, sms);
    p.tpr = t.tpr;
    const int slots = t.slots, threads = t.per * t.tpr;
    const long long ctas = std::min((p.rows + t.per - 1) / t.per, static_cast<long long>(sms) * std::max<long long>(1, t.room / threads));
    void (*const fn)(const NormParams) = !full && CODES ? (vec ? norm_of<T, true, true, false>(slots) : norm_of<T, true, false, false>(slots))
                                                        : (vec ? norm_of<T, CODES, true, true>(slots) : norm_of<T, CODES, false, true>(slots));
    return launched("norm", launch_behind(fn, p, dim3(static_cast<unsigned>(ctas)), threads, st));
}

template <class T>
spec_status norm_as(const NormParams& p, bool codes, int B, cudaStream_t st) {
    const int sms = sm_count();
    if (sms < 1) return fail(SPEC_ERR_CUDA, "device query failed");
    const bool vec = whole_pieces(p, sizeof(T), codes, B);
    const bool peel = !vec && alike_rows(p, sizeof(T), codes, B);
    return codes ? norm_as<T, true>(p, vec, peel, sms, st) : norm_as<T, false>(p, vec, peel, sms, st);
}

spec_status norm(const NormParams& p, int dtype, bool codes, int B, cudaStream_t st) {
    return dtype == SPEC_BF16 ? norm_as<__nv_bfloat16>(p, codes, B, st)
           : dtype == SPEC_FP16 ? norm_as<__half>(p, codes, B, st) : norm_as<float>(p, codes, B, st);
}

spec_status check_norm(int dtype, int B, int N, int D) {
    SPECS_TRY(check_type(dtype));
    SPECS_TRY(check_tokens(B, N));
    if (D < 1 || D > SPEC_SCORE_MAX_D)
        return fail(SPEC_ERR_UNSUPPORTED, "D must be in [1, %d], got %d", SPEC_SCORE_MAX_D, D);
    return SPEC_OK;
}

// --------------------------------------------------------------------------------------------- product
// Workspace: header, and the tokens' halves in tiles of equal width, a multiple of 32.
size_t matmul_bytes(int tokens, int, int K) {
    const size_t tiles = (static_cast<size_t>(tokens) + PR_TOKENS - 1) / PR_TOKENS;
    return SPEC_SCORE_WS_HEADER + ((static_cast<size_t>(tokens) + 31) / 32 * 32 + 32 * tiles) * ((static_cast<size_t>(K) + PR_K - 1) / PR_K * PR_K) * 2;
}

template <class T, bool ALIGNED>
spec_status matvec_as(MatmulParams p, cudaStream_t st) {
    // as few warps to a channel's K as still give every SM its 64: then each has more loads on their way and fewer sums to join
    p.k_warps = 1;
    while (p.k_warps < 8 && p.K > 512 * p.k_warps && static_cast<long long>((p.C + MV_CH - 1) / MV_CH) * p.k_warps < 48LL * MV_SMS) p.k_warps *= 2;
    const int per = MV_WARPS / p.k_warps * MV_CH;
    const int width = p.tokens > 4 ? 8 : p.tokens > 2 ? 4 : p.tokens;
    void (*const fn)(const MatmulParams) = width == 8 ? matvec_kernel<T, 8, ALIGNED> : width == 4 ? matvec_kernel<T, 4, ALIGNED>
                                           : width == 2 ? matvec_kernel<T, 2, ALIGNED> : matvec_kernel<T, 1, ALIGNED>;
    return launched("product", launch_behind(fn, p, dim3((p.C + per - 1) / per), MV_WARPS * 32, st));
}

template <class T>
spec_status matvec(const MatmulParams& p, bool aligned, cudaStream_t st) {
    return aligned ? matvec_as<T, true>(p, st) : matvec_as<T, false>(p, st);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
    static std::atomic<void*> found{nullptr};
    void* f = found.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult how;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &how) != cudaSuccess ||
            how != cudaDriverEntryPointSuccess)
            return nullptr;
        found.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

template <class T, bool PAIR, bool MAP, bool HERE = false>
spec_status product_as(const ProductParams& p, int grid, cudaStream_t st) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(SPEC_ERR_CUDA, "device query failed");
    static std::atomic<unsigned> ready{0};       // devices whose limit of dynamic shared memory is raised
    const unsigned bit = dev < 32 ? 1u << dev : 0u;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(product_kernel<T, PAIR, MAP, HERE>, cudaFuncAttributeMaxDynamicSharedMemorySize, PR_SMEM);
        if (e != cudaSuccess) return fail(SPEC_ERR_CUDA, "product kernel attribute failed: %s", cudaGetErrorString(e));
        ready.fetch_or(bit, std::memory_order_release);
    }
    return launched("product", launch_behind(product_kernel<T, PAIR, MAP, HERE>, p, dim3(grid), PR_THREADS, st, PR_SMEM, PAIR ? 2 : p.split));
}

spec_status product(const MatmulParams& m, bool map, bool a16, int out_type, unsigned char* ws, cudaStream_t st) {
    const int sms = sm_count();
    if (sms < 1) return fail(SPEC_ERR_CUDA, "device query failed");
    ProductParams p = {};
    if (map) {
        const EncodeTiled encode = encode_tiled();
        if (!encode) return fail(SPEC_ERR_CUDA, "cuTensorMapEncodeTiled is not to be had");
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(m.K), static_cast<cuuint64_t>(m.C)};
        const cuuint64_t strides[1] = {m.C > 1 ? static_cast<cuuint64_t>(m.w_stride) : static_cast<cuuint64_t>((m.K + 15) / 16 * 16)};
        const cuuint32_t box[2] = {PR_K, PR_CH}, one[2] = {1, 1};
        if (encode(&p.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<signed char*>(m.w), dims, strides, box, one,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return fail(SPEC_ERR_CUDA, "no tensor map for w");
    }
    p.codes = m.w;
    p.w_stride = m.w_stride;
    p.K = m.K;
    p.out = m.out;
    p.tokens16 = ws + SPEC_SCORE_WS_HEADER;
    p.a_scale = m.a_scale;
    p.w_scale = m.w_scale;
    p.bias = m.bias;
    p.tokens = m.tokens;
    p.N = m.N;
    p.C = m.C;
    p.steps = (m.K + PR_K - 1) / PR_K;
    p.status = reinterpret_cast<unsigned*>(ws);
    p.token_tiles = (m.tokens + PR_TOKENS - 1) / PR_TOKENS;
    const bool pair = map && m.tokens > 64 && static_cast<long long>((m.C + 2 * PR_CH - 1) / (2 * PR_CH)) * p.token_tiles >= sms / 4;
    if (!pair) p.token_tiles = (m.tokens + PR_TOKENS_ALONE - 1) / PR_TOKENS_ALONE;
    const int per = (m.tokens + p.token_tiles - 1) / p.token_tiles;
    p.n = pair ? (per + 31) / 32 * 32 : (per + 15) / 16 * 16;
    p.channel_tiles = (m.C + PR_CH * (pair ? 2 : 1) - 1) / (PR_CH * (pair ? 2 : 1));
    const long long units = static_cast<long long>(p.channel_tiles) * p.token_tiles;
    if (units > (1LL << 30)) return fail(SPEC_ERR_UNSUPPORTED, "too many tokens and channels: %lld tiles", units);
    p.split = 1;
    if (!pair)
        while (p.split < 8 && units * p.split * 2 <= sms && p.split * 2 <= p.steps) p.split *= 2;
    p.stages = std::min(PR_STAGES, (PR_SMEM - 1024) / (PR_W_BYTES + 2 * 128 * (pair ? p.n / 2 : p.n)));
    if (p.stages < PR_MIN_STAGES) return fail(SPEC_ERR_CUDA, "no room for %d stages", PR_MIN_STAGES);
    p.stream_w = p.token_tiles <= 8;
    // Up to 32 tokens of few weights become halves where they are used: a CTA does that for each of its channel tiles, but there is
    // one launch less. In us, so / in a kernel of their own: 16 tokens over 1024 x 1024 5.1 and 6.7, 4096 x 4096 8.9 and 10.2, 14336 x
    // 4096 18.8 and 18.4, 128256 x 4096 109 and 96; 32 tokens over 4096 x 4096 10.0 and 11.1, 14336 x 4096 19.5 and 18.5.
    const bool here = map && a16 && m.tokens <= 32 && static_cast<long long>(m.C) * m.K <= 32000000LL;
    p.a = m.a;
    HalvesParams h = {};
    h.a = m.a;
    h.out = ws + SPEC_SCORE_WS_HEADER;
    h.tokens = m.tokens;
    h.N = m.N;
    h.K = m.K;
    h.n = p.n;
    h.steps = p.steps;
    h.groups = static_cast<long long>(p.token_tiles) * p.n * p.steps * (PR_K / 16);
    if (!here) SPECS_TRY(launched("product's halves", launch_behind(halves_kernel, h, dim3(static_cast<unsigned>((h.groups + 255) / 256)), 256, st)));
    if (pair) {
        const int grid = static_cast<int>(std::min<long long>(units, sms / 2)) * 2;
        return out_type == SPEC_BF16 ? product_as<__nv_bfloat16, true, true>(p, grid, st)
               : out_type == SPEC_FP16 ? product_as<__half, true, true>(p, grid, st) : product_as<float, true, true>(p, grid, st);
    }
    const int grid = p.split > 1 ? static_cast<int>(units) * p.split : static_cast<int>(std::min<long long>(units, sms));
    if (here)
        return out_type == SPEC_BF16 ? product_as<__nv_bfloat16, false, true, true>(p, grid, st)
               : out_type == SPEC_FP16 ? product_as<__half, false, true, true>(p, grid, st) : product_as<float, false, true, true>(p, grid, st);
    if (map)
        return out_type == SPEC_BF16 ? product_as<__nv_bfloat16, false, true>(p, grid, st)
               : out_type == SPEC_FP16 ? product_as<__half, false, true>(p, grid, st) : product_as<float, false, true>(p, grid, st);
    return out_type == SPEC_BF16 ? product_as<__nv_bfloat16, false, false>(p, grid, st)
           : out_type == SPEC_FP16 ? product_as<__half, false, false>(p, grid, st) : product_as<float, false, false>(p, grid, st);
}

// ---------------------------------------------------------------------------------------------- logits
template <class T, bool MASK>
spec_status logits_as(const LogitsParams& p, int B, cudaStream_t st) {
    const size_t smem = (static_cast<size_t>(p.seg) + p.seg / 32 + 16) * 4;
    static_assert((LG_SEG + LG_SEG / 32 + 16) * 4 <= 40 * 1024, "within what every kernel may have");
    return launched("logits", launch_behind(logits_kernel<T, MASK>, p, dim3((p.V + p.seg - 1) / p.seg, B), LG_THREADS, st, smem));
}

}  // namespace
}  // namespace specs

using namespace specs;

extern "C" {

const char* spec_score_last_error(void) { return g_err; }

spec_status spec_residual_norm(const spec_rows* x, const spec_rows* residual, int dtype, int B, int N, int D,
                               const void* weight, float eps, const spec_rows* residual_out, const spec_rows* out,
                               int out_type, float* scale, void* stream) {
    SPECS_TRY(check_norm(dtype, B, N, D));
    if (out_type != SPEC_INT8 && out_type != dtype)
        return fail(SPEC_ERR_UNSUPPORTED, "out_type must be dtype or SPEC_INT8, got %d", out_type);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(SPEC_ERR_INVALID, "eps must be finite and not negative");
    if (!residual != !residual_out) return fail(SPEC_ERR_INVALID, "residual and residual_out come together");
    if (B == 0 || N == 0) return SPEC_OK;
    const size_t e = type_bytes(dtype);
    SPECS_TRY(check_rows(x, "x", e));
    if (residual) {
        SPECS_TRY(check_rows(residual, "residual", e));
        SPECS_TRY(check_out(residual_out, "residual_out", e, B, N, D));
    }
    SPECS_TRY(check_out(out, "out", type_bytes(out_type), B, N, D));
    if (residual && residual_out->data == out->data) return fail(SPEC_ERR_INVALID, "out must not be residual_out");
    if (residual) SPECS_TRY(check_same(residual_out, "residual_out", x, residual, B, N));
    if (out_type != SPEC_INT8) SPECS_TRY(check_same(out, "out", x, residual, B, N));
    else if (out->data == x->data || (residual && out->data == residual->data))
        return fail(SPEC_ERR_INVALID, "out in 8 bits must not be an input");
    if (out_type == SPEC_INT8 && !scale) return fail(SPEC_ERR_INVALID, "scale must not be NULL");
    SPECS_TRY(check_words({{scale, "scale"}}));
    if (reinterpret_cast<uintptr_t>(weight) % e) return fail(SPEC_ERR_INVALID, "weight: the pointer must be a multiple of %zu bytes", e);
    NormParams p = {};
    p.x = rows_of(x);
    p.res = rows_of(residual);
    p.res_out = rows_of(residual_out);
    p.out = rows_of(out);
    p.weight = weight;
    p.scale = scale;
    p.rows = static_cast<long long>(B) * N;
    p.N = N;
    p.D = D;
    p.eps = eps;
    p.norm = 1;
    return norm(p, dtype, out_type == SPEC_INT8, B, static_cast<cudaStream_t>(stream));
}

spec_status spec_quantize_rows(const spec_rows* x, int dtype, int B, int N, int D, const spec_rows* out, float* scale,
                               void* stream) {
    SPECS_TRY(check_norm(dtype, B, N, D));
    if (B == 0 || N == 0) return SPEC_OK;
    SPECS_TRY(check_rows(x, "x", type_bytes(dtype)));
    SPECS_TRY(check_out(out, "out", 1, B, N, D));
    if (out->data == x->data) return fail(SPEC_ERR_INVALID, "out in 8 bits must not be an input");
    if (!scale) return fail(SPEC_ERR_INVALID, "scale must not be NULL");
    SPECS_TRY(check_words({{scale, "scale"}}));
    NormParams p = {};
    p.x = rows_of(x);
    p.out = rows_of(out);
    p.scale = scale;
    p.rows = static_cast<long long>(B) * N;
    p.N = N;
    p.D = D;
    return norm(p, dtype, true, B, static_cast<cudaStream_t>(stream));
}

size_t spec_int8_matmul_workspace_size(int tokens, int C, int K) {
    if (tokens < 0 || tokens > MAX_TOKENS || C < 0 || C > MAX_C || K < 1 || K > SPEC_SCORE_MAX_K) return 0;
    return matmul_bytes(tokens, C, K);
}

spec_status spec_int8_matmul(const spec_rows* a, const float* a_scale, const void* w, long long w_stride,
                             const float* w_scale, const float* bias, int B, int N, int C, int K, const spec_rows* out,
                             int out_type, void* workspace, size_t workspace_bytes, void* stream) {
    SPECS_TRY(check_type(out_type));
    SPECS_TRY(check_tokens(B, N));
    if (C < 0 || C > MAX_C) return fail(SPEC_ERR_INVALID, "C must be in [0, %d], got %d", MAX_C, C);
    if (K < 1 || K > SPEC_SCORE_MAX_K) return fail(SPEC_ERR_UNSUPPORTED, "K must be in [1, %d], got %d", SPEC_SCORE_MAX_K, K);
    if (B == 0 || N == 0 || C == 0) return SPEC_OK;
    SPECS_TRY(check_rows(a, "a", 1));
    SPECS_TRY(check_out(out, "out", type_bytes(out_type), B, N, C));
    if (!w || !a_scale || !w_scale) return fail(SPEC_ERR_INVALID, "w, a_scale and w_scale must not be NULL");
    SPECS_TRY(check_words({{a_scale, "a_scale"}, {w_scale, "w_scale"}, {bias, "bias"}}));
    if (C > 1 && w_stride < 0) return fail(SPEC_ERR_INVALID, "w_stride must not be negative");
    if (!workspace || !aligned16(workspace)) return fail(SPEC_ERR_INVALID, "workspace must be 16-byte aligned device memory");
    const size_t need = matmul_bytes(B * N, C, K);
    if (workspace_bytes < need) return fail(SPEC_ERR_INVALID, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
    MatmulParams p = {};
    p.a = rows_of(a);
    p.out = rows_of(out);
    p.w = static_cast<const signed char*>(w);
    p.a_scale = a_scale;
    p.w_scale = w_scale;
    p.bias = bias;
    p.w_stride = w_stride;
    p.tokens = B * N;
    p.N = N;
    p.C = C;
    p.K = K;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // what a tensor map can hold: rows on 16 bytes that do not overlap
    const bool codes16 = aligned16(w) && (C == 1 || (w_stride % 16 == 0 && w_stride >= K && w_stride < (1LL << 40)));
    // Up to eight tokens of not too many weights go without the tensor cores, whose two kernels take 6 us before they are under way. In
    // us, this way / with tensor cores (C x K):
    //   tokens  1024 x 4096   4096 x 4096   14336 x 4096   8192 x 8192   128256 x 4096
    //   1       2.3  7.1      4.0  9.5      12.3  18.2     12.6  19.3    78.4   96.8
    //   2       2.1  7.1      4.2  9.6      13.1  18.2     13.5  19.4    82.7   96.9
    //   4       3.0  7.2      5.8  9.5      18.1  18.2     22.3  19.4    99.9   96.4
    //   8       3.4  7.3      9.7  9.6      24.5  18.2     22.4  19.9    124.7  96.6
    const long long weights = static_cast<long long>(C) * K;
    // Rows off 16 bytes: 8 tokens, 14336 x 4099: 62 and 104; 64 tokens, 2000 x 4097: 77 and 27.
    const bool few = p.tokens <= 2 || (p.tokens <= 8 && (!codes16 || weights <= (p.tokens <= 4 ? 50000000LL : 16000000LL)));
    const bool a16 = K % 16 == 0 && aligned16(a->data) && (B == 1 || a->stride_b % 16 == 0) && (N == 1 || a->stride_n % 16 == 0);
    if (!few) return product(p, codes16, a16, out_type, static_cast<unsigned char*>(workspace), st);
    const bool aligned = a16 && aligned16(w) && (C == 1 || w_stride % 16 == 0);
    return out_type == SPEC_BF16   ? matvec<__nv_bfloat16>(p, aligned, st)
           : out_type == SPEC_FP16 ? matvec<__half>(p, aligned, st) : matvec<float>(p, aligned, st);
}

spec_status spec_process_logits(const spec_rows* logits, int dtype, int B, int R, int V, const int32_t* tokens, int T,
                                const int32_t* history, const int32_t* lengths, const int32_t* prompt, int L,
                                const float* repetition, const float* frequency, const float* presence,
                                const int32_t* bias_tokens, const float* bias, int biases, const uint32_t* mask,
                                long long mask_stride_b, long long mask_stride_r, const spec_rows* out, void* stream) {
    if (dtype != SPEC_BF16 && dtype != SPEC_FP32) return fail(SPEC_ERR_UNSUPPORTED, "dtype must be bf16 or fp32, got %d", dtype);
    if (B < 0 || B > MAX_B) return fail(SPEC_ERR_INVALID, "B must be in [0, %d], got %d", MAX_B, B);
    if (R < 0 || R > SPEC_SCORE_MAX_ROWS) return fail(SPEC_ERR_INVALID, "R must be in [0, %d], got %d", SPEC_SCORE_MAX_ROWS, R);
    if (V < 1 || V > MAX_V) return fail(SPEC_ERR_INVALID, "V must be in [1, %d], got %d", MAX_V, V);
    if (L < 0 || L > SPEC_SCORE_MAX_HISTORY) return fail(SPEC_ERR_INVALID, "L must be in [0, %d], got %d", SPEC_SCORE_MAX_HISTORY, L);
    if (biases < 0 || biases > SPEC_SCORE_MAX_BIASES)
        return fail(SPEC_ERR_INVALID, "biases must be in [0, %d], got %d", SPEC_SCORE_MAX_BIASES, biases);
    if (B == 0 || R == 0) return SPEC_OK;
    const size_t e = type_bytes(dtype);
    SPECS_TRY(check_rows(logits, "logits", e));
    SPECS_TRY(check_out(out, "out", e, B, R, V));
    SPECS_TRY(check_same(out, "out", logits, nullptr, B, R));
    if (tokens && T < R - 1) return fail(SPEC_ERR_INVALID, "tokens must have at least R - 1 = %d a sequence, got %d", R - 1, T);
    if (history && L > 0 && !lengths) return fail(SPEC_ERR_INVALID, "lengths must not be NULL");
    if (bias_tokens && biases > 0 && !bias) return fail(SPEC_ERR_INVALID, "bias must not be NULL");
    SPECS_TRY(check_words({{tokens, "tokens"}, {history, "history"}, {lengths, "lengths"}, {prompt, "prompt"}, {repetition, "repetition"},
                           {frequency, "frequency"}, {presence, "presence"}, {bias_tokens, "bias_tokens"}, {bias, "bias"}, {mask, "mask"}}));
    LogitsParams p = {};
    p.in = rows_of(logits);
    p.out = rows_of(out);
    p.tokens = tokens;
    p.history = L > 0 ? history : nullptr;
    p.lengths = lengths;
    p.prompt = prompt;
    p.bias_tokens = biases > 0 ? bias_tokens : nullptr;
    p.repetition = repetition;
    p.frequency = frequency;
    p.presence = presence;
    p.bias = bias;
    p.mask = mask;
    p.mask_sb = mask_stride_b;
    p.mask_sr = mask_stride_r;
    p.R = R;
    p.V = V;
    p.T = T;
    p.L = L;
    p.biases = biases;
    const int sms = sm_count();
    if (sms < 1) return fail(SPEC_ERR_CUDA, "device query failed");
    // as large a part of the vocabulary as still gives the card four CTAs an SM: each reads the whole history
    p.seg = LG_SEG;
    while (p.seg > 1024 && static_cast<long long>((V + p.seg - 1) / p.seg) * B < 4LL * sms) p.seg /= 2;
    auto alike = [&](long long x, long long y) { return (x - y) * static_cast<long long>(e) % 16 == 0; };
    p.pieces = (reinterpret_cast<uintptr_t>(logits->data) - reinterpret_cast<uintptr_t>(out->data)) % 16 == 0 &&
               (B == 1 || alike(logits->stride_b, out->stride_b)) && (R == 1 || alike(logits->stride_n, out->stride_n));
    p.together = p.pieces && (R == 1 || alike(logits->stride_n, 0));
    p.stream = out->data != logits->data || mask;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (mask) return dtype == SPEC_BF16 ? logits_as<__nv_bfloat16, true>(p, B, st) : logits_as<float, true>(p, B, st);
    return dtype == SPEC_BF16 ? logits_as<__nv_bfloat16, false>(p, B, st) : logits_as<float, false>(p, B, st);
}

}  // extern "C"
