// The product of 8-bit integers on the tensor cores, which take no 8-bit integers on this card: as halves, exactly.
#pragma once
#include <cuda.h>

#include "../cache/tmem.cuh"
#include "matmul.cuh"

namespace specs {

using specv::smem_addr;

// A step is 128 of K: 128 channels' codes as they are (16 KB) and the tokens' halves.
constexpr int PR_K = 128, PR_CH = 128, PR_TOKENS = 192, PR_THREADS = 640, PR_STAGES = 11;
// Warps that turn step g's codes wait for its copies when they have written step g - 2, so when the products of step g - 4 are
// done: the stage's barrier is then in the phase that they mean only if its last use was no later than that.
constexpr int PR_MIN_STAGES = 4, PR_TOKENS_ALONE = 128;      // a CTA without a pair has room for four stages up to 144 tokens
constexpr int PR_W_BYTES = PR_CH * PR_K;
constexpr int PR_SMEM = 222 * 1024;                    // of it up to 1 KB is lost to alignment
constexpr uint32_t PR_COL_A = 2 * PR_TOKENS;           // tensor memory: two accumulators, two steps of channels
constexpr uint64_t PR_WAIT_NS = 2000000000ull;
// The sum of four steps is at most 512 x 2^14 = 2^23 in magnitude, so exact in fp32 as are its parts.
constexpr int PR_CHUNK = 4;

struct ProductParams {
    CUtensorMap w;       // 64-byte aligned, as its type says
    Rows out;
    const unsigned char* tokens16;
    const float *a_scale, *w_scale, *bias;
    Rows a;                        // the tokens' codes, where they become halves here
    const signed char* codes;      // w, for rows that no tensor map can hold
    long long w_stride;
    int tokens, N, C, K;
    int n, token_tiles, channel_tiles, steps, stages, split;
    int stream_w;        // the codes are read once: they need not stay in L2
    unsigned* status;
};

struct HalvesParams {
    Rows a;
    unsigned char* out;
    int tokens, N, K, n, steps;
    long long groups;    // of 16 codes
};

// ------------------------------------------------------------------------------------ tokens to halves
// The tokens' codes as halves, in the blocks that the product reads: for each tile of n tokens and 64 of K, n rows of 128 bytes
// whose 16-byte pieces are exchanged as 128-byte swizzling wants it (piece c of row r at c ^ (r & 7)). Rows and columns past the
// ends are 0. A few MB from and to L2; the product's first copies of codes are on their way meanwhile.
__device__ __forceinline__ void halves_of(uint32_t x, uint32_t& lo, uint32_t& hi) {
    // a byte b behind 0x64 is the half 1024 + b; with b = code + 128 that is the code and 1152
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    x ^= 0x80808080u;
    const uint32_t l = __byte_perm(x, 0x64646464u, 0x4140), h = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), off), b = __hsub2(*reinterpret_cast<const __half2*>(&h), off);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
}

__global__ void __launch_bounds__(256) halves_kernel(const __grid_constant__ HalvesParams p) {
    after_previous();
    const long long g = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (g >= p.groups) return;
    const int per_row = p.steps * (PR_K / 16);
    const int row = static_cast<int>(g / per_row), k = static_cast<int>(g - static_cast<long long>(row) * per_row) * 16;
    uint32_t x[4] = {0u, 0u, 0u, 0u};
    if (row < p.tokens && k < p.K) {
        const signed char* const src = row_of<signed char>(p.a, row / p.N, row % p.N) + k;
        if (k + 16 <= p.K && (reinterpret_cast<uintptr_t>(src) & 15) == 0) {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (k + i < p.K) x[i / 4] |= static_cast<uint32_t>(static_cast<unsigned char>(src[i])) << (8 * (i % 4));
        }
    }
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) halves_of(x[i], h[2 * i], h[2 * i + 1]);
    const int tile = row / p.n, r = row - tile * p.n, c = k % 64 / 8;
    unsigned char* const dst = p.out + (static_cast<long long>(tile) * p.steps * 2 + k / 64) * p.n * 128 + r * 128;
    *reinterpret_cast<uint4*>(dst + ((c ^ (r & 7)) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(dst + (((c + 1) ^ (r & 7)) * 16)) = make_uint4(h[4], h[5], h[6], h[7]);
}

// ------------------------------------------------------------------------------------------- the product
__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits, as a warp, for a phase of `bar`. A lane that gives up sets the status bit and clears its `alive`, so that its later waits end
// at once: the results are invalid, but every barrier behind is still met.
__device__ __forceinline__ void wait_phase(uint64_t* bar, uint32_t parity, bool& alive, unsigned* status) {
    uint64_t since = 0;
    for (int i = 1; !phase_done(bar, parity) && alive; ++i) {
        if (i % 256 == 0) {
            const uint64_t now = specv::global_timer_ns();
            if (since == 0) since = now;
            if (now - since >= PR_WAIT_NS) {
                atomicOr(status, SPEC_STATUS_TIMEOUT);
                alive = false;
            }
        }
    }
    __syncwarp();
}

// Whether the phase is over, without a wait.
__device__ __forceinline__ bool phase_over(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Arrives at the barrier of the pair's first CTA (its own one where there is no pair).
template <bool PAIR>
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
            "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_addr(bar))
            : "memory");
    else
        specv::mbar_arrive(bar);
}

// Of the lane with `lead`, in converged code: so the operands stay where the warp's common values are.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t lead) {      // at both CTAs of a pair
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(smem_addr(bar)),
            "h"(static_cast<unsigned short>(3)), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)), "r"(lead)
            : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t lead) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
            "r"(static_cast<uint32_t>(add)), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
            "r"(static_cast<uint32_t>(add)), "r"(lead)
            : "memory");
}

__device__ __forceinline__ void load_codes(void* dst, const CUtensorMap* map, int k, int channel, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(k), "r"(channel), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

// Tokens' halves in shared memory: rows of 128 bytes, swizzled, eight rows to 1024 bytes; `addr` in 16 bytes.
__device__ __forceinline__ uint64_t tokens_desc(uint32_t addr) {
    return static_cast<uint64_t>(addr & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <int REGS, bool MORE>
__device__ __forceinline__ void set_registers() {
    if (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// The units of a CTA (a pair): tiles of channels times tiles of tokens. Tiles of tokens come in groups of eight, within which the
// units of neighbouring CTAs share their channels' codes.
struct Unit {
    int channel, tile;
    __device__ Unit(const ProductParams& p, int u) {
        const int per = 8 * p.channel_tiles, group = u / per, wide = min(8, p.token_tiles - 8 * group), in = u - group * per;
        channel = in / wide;
        tile = 8 * group + in % wide;
    }
};

// Channels stand on the tensor cores' long side, tokens on the other. Four parts work beside one another:
//   warp 0         copies: the channels' codes as they are in memory, the tokens' halves
//   warp 1         products: D[channel, token] += A[channel, k] B[k, token], A in tensor memory, 16 of K at a time
//   warps 4 .. 11  codes to halves, exactly, from shared to tensor memory; two halves of the warps take the steps in turn
//   warps 12 .. 19 sums of 512 products out of the tensor memory into integers in registers, and at the end to the output; each half
//                  of the warps takes half of the tokens
// PAIR: two CTAs share a tile of 256 channels; each holds its channels and half of the tokens, the first one issues.
// MAP: the codes' rows are on 16 bytes, and copies bring them; else the warps that turn them fetch them themselves, 16 bytes a lane.
// HERE: up to 32 tokens, one tile of them, whose codes the same warps fetch and turn, a step of theirs ahead: one launch.
// split > 1: the CTAs of a cluster share a tile's K, and add their integers through one another's shared memory.
// A few passes behind one another, 384 tokens over 128256 channels of 4096 take 246 us, 1.64 P operations a second, 84% of what a library
// product in bf16 reaches in a burst; 8192 tokens over 14336 channels of 4096 550 us, 90%. Launched for seconds on end, under the power
// limit, 270 and 603 us, 85% and 91% of what the library sustains. 384 tokens over a layer's 14336 x 4096 take 39.5 us (C x K), over
// 4096 x 14336 54.2, over 4096 x 4096 20.5; the floors are 23.2, 23.2 and 6.6.
template <class T, bool PAIR, bool MAP, bool HERE>
__global__ void __launch_bounds__(PR_THREADS, 1) product_kernel(const __grid_constant__ ProductParams p) {
    extern __shared__ unsigned char dynamic[];
    __shared__ alignas(8) uint64_t s_full[PR_STAGES], s_empty[PR_STAGES], s_ready[4], s_half_empty[2], s_acc_full[2], s_acc_empty[2];
    __shared__ uint32_t s_tmem;
    __shared__ alignas(16) float s_scales[2][PR_TOKENS];
    __shared__ alignas(16) long long s_rows[2][PR_TOKENS];      // of this tile and the next
    unsigned char* const smem = dynamic + ((1024u - (smem_addr(dynamic) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    constexpr int CTAS = PAIR ? 2 : 1;
    const int rank = PAIR || p.split > 1 ? static_cast<int>(specv::cluster_ctarank()) : 0;
    const int own_n = p.n / CTAS, half_bytes = own_n * 128, stage_bytes = PR_W_BYTES + 2 * half_bytes;
    const int group = PAIR ? 2 : p.split;
    const int units = p.channel_tiles * p.token_tiles, first = blockIdx.x / group, by = gridDim.x / group;      // the host keeps units small
    const int k_from = PAIR ? 0 : static_cast<int>(static_cast<long long>(p.steps) * rank / p.split);
    const int k_to = PAIR ? p.steps : static_cast<int>(static_cast<long long>(p.steps) * (rank + 1) / p.split);
    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) specv::mbar_init(&s_full[i], 1), specv::mbar_init(&s_empty[i], 1);
        for (int i = 0; i < 4; ++i) specv::mbar_init(&s_ready[i], 4 * CTAS);
        for (int i = 0; i < 2; ++i) specv::mbar_init(&s_half_empty[i], 1), specv::mbar_init(&s_acc_full[i], 1), specv::mbar_init(&s_acc_empty[i], 8 * CTAS);
        specv::fence_mbarrier_init_cluster();
    }
    if (warp == 2) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&s_tmem)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            specc::tmem_alloc(&s_tmem, 512);
        }
        specc::tmem_fence_before();
    }
    __syncthreads();
    if (PAIR) specv::cluster_sync_all();
    specc::tmem_fence_after();
    const uint32_t tmem = s_tmem;
    bool alive = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { wait_phase(bar, parity, alive, p.status); };

    if (warp < 4) {
        set_registers<48, false>();
        if (warp == 0) {
            // ================ copies
            const uint64_t keep = specv::policy_evict_last(), w_policy = p.stream_w ? specv::policy_evict_first() : specv::policy_evict_normal();
            auto codes = [&](int st, const Unit& u, int k) {
                if (lane == 0) {
                    specv::mbar_arrive_expect_tx(&s_full[st], (MAP ? PR_W_BYTES : 0) + (HERE ? 0 : 2 * half_bytes));
                    if (MAP) load_codes(smem + st * stage_bytes, &p.w, k * PR_K, (u.channel * CTAS + (PAIR ? rank : 0)) * PR_CH, &s_full[st], w_policy);
                }
            };
            auto tokens = [&](int st, const Unit& u, int k) {
                if (!HERE && lane < 2) {
                    const unsigned char* src = p.tokens16 + ((static_cast<long long>(u.tile) * p.steps + k) * 2 + lane) * p.n * 128 + (PAIR ? rank * half_bytes : 0);
                    specv::bulk_load(smem + st * stage_bytes + PR_W_BYTES + lane * half_bytes, src, half_bytes, &s_full[st], keep);
                }
            };
            // The first copies of codes are on their way before the kernel in front, which makes the tokens' halves, has ended: what
            // it waited for before it let this one in holds the codes.
            int ahead = 0;
            if (HERE) asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");      // no kernel in front
            if (first < units) {
                const Unit u(p, first);
                for (; ahead < p.stages && k_from + ahead < k_to; ++ahead) codes(ahead, u, k_from + ahead);
            }
            if (!HERE) asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
            int g = 0, st = 0;
            uint32_t round = 0;      // of the stages' uses
            for (int i = first; i < units; i += by) {
                const Unit u(p, i);
                for (int k = k_from; k < k_to; ++k) {
                    if (g >= ahead) {
                        if (round > 0) wait(&s_empty[st], (round - 1) & 1);
                        if (alive) codes(st, u, k);
                    }
                    __syncwarp();
                    if (alive) tokens(st, u, k);
                    ++g;
                    if (++st == p.stages) st = 0, ++round;
                }
            }
            // this CTA's copies have landed, and the products' arrivals are in, before it ends
            for (int i = max(0, g - p.stages); i < g; ++i) {
                bool once = alive;
                wait_phase(&s_full[i % p.stages], (i / p.stages) & 1, once, p.status);
                wait(&s_empty[i % p.stages], (i / p.stages) & 1);
            }
        } else if (warp == 1 && (!PAIR || rank == 0)) {
            // ================ products, issued by one lane
            // a kernel in front that lasts does not count as this one's wait
            if (HERE) asm volatile("griddepcontrol.wait;" ::: "memory");
            const uint32_t lead = specc::elect_one();
            const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(p.n >> 3) << 17) | (static_cast<uint32_t>(PR_CH * CTAS >> 4) << 24);
            const uint32_t base = smem_addr(smem + PR_W_BYTES) >> 4, half = half_bytes >> 4;
            int st = 0, chunk = 0;
            uint32_t at = 0;                                         // half steps
            bool over = phase_over(&s_ready[0], 0);                  // looked at one half step ahead
            for (int i = first; i < units; i += by)
                for (int k = k_from; k < k_to; ++k) {
                    const bool starts = (k - k_from) % PR_CHUNK == 0, ends = (k - k_from) % PR_CHUNK == PR_CHUNK - 1 || k + 1 == k_to;
                    const uint32_t d = tmem + (chunk & 1) * PR_TOKENS, b = base + st * (stage_bytes >> 4);
                    if (starts && chunk >= 2) wait(&s_acc_empty[chunk & 1], ((chunk >> 1) - 1) & 1);
#pragma unroll
                    for (int h = 0; h < 2; ++h, ++at) {
                        if (!__all_sync(0xffffffffu, over)) wait(&s_ready[at & 3], (at >> 2) & 1);
                        specc::tmem_fence_after();
                        over = phase_over(&s_ready[(at + 1) & 3], ((at + 1) >> 2) & 1);
                        const uint32_t a = tmem + PR_COL_A + (at & 3) * 32, go = alive ? lead : 0u;
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma<PAIR>(d, a + 8 * j, tokens_desc(b + h * half + j * 2), idesc, !starts || h > 0 || j > 0, go);
                        commit<PAIR>(h ? &s_empty[st] : &s_half_empty[(at >> 1) & 1], go);
                        if (h && ends) commit<PAIR>(&s_acc_full[chunk & 1], go);
                    }
                    if (ends) ++chunk;
                    if (++st == p.stages) st = 0;
                }
        }
    } else if (warp < 12) {
        // ================ codes to halves
        set_registers<80, false>();
        const int mine = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t to = tmem + PR_COL_A + mine * 64 + (static_cast<uint32_t>(warp & 3) << 21);
        // HERE: the lane's tokens, eight lanes to a row's 16 bytes each, and their codes for this buffer's next step
        const int t = tid & 127, piece = t & 7;
        const signed char* token[2] = {nullptr, nullptr};
        uint4 codes[2];
        auto fetch = [&](int k) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                codes[r] = make_uint4(0u, 0u, 0u, 0u);
                if (token[r] && k * PR_K + piece * 16 < p.K) codes[r] = __ldg(reinterpret_cast<const uint4*>(token[r] + k * PR_K + piece * 16));
            }
        };
        if (HERE) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int n = r * 16 + (t >> 3), b = n / p.N;
                if (n < p.tokens) token[r] = row_of<const signed char>(p.a, b, n - b * p.N);
            }
            fetch(k_from + mine % (k_to - k_from));
        }
        int g = 0, st = -1, used = -1;      // step, its stage, the stage of this buffer's last step
        uint32_t round = 0, used_round = 0;
        for (int i = first; i < units; i += by)
            for (int k = k_from; k < k_to; ++k, ++g) {
                if (++st == p.stages) st = 0, ++round;
                if ((g & 1) != mine) continue;
                if constexpr (!MAP) {
                    // eight lanes to a row's 128 codes; the place in shared memory is free when the step's other copies may begin
                    unsigned char* const to_row = smem + st * stage_bytes;
                    const int at = k * PR_K + piece * 16;
                    const Unit u(p, i);
                    int x[8][4];
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const int c = u.channel * PR_CH + r * 16 + (t >> 3);
                        x[r][0] = x[r][1] = x[r][2] = x[r][3] = 0;
                        if (c < p.C && at < p.K) load16<false>(p.codes + c * p.w_stride + at, p.K - at, x[r]);
                    }
                    wait(&s_full[st], round & 1);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const int c = r * 16 + (t >> 3);
                        *reinterpret_cast<int4*>(to_row + c * 128 + ((piece ^ (c & 7)) * 16)) = make_int4(x[r][0], x[r][1], x[r][2], x[r][3]);
                    }
                    asm volatile("bar.sync %0, 128;" ::"r"(2 + mine) : "memory");
                } else {
                    wait(&s_full[st], round & 1);
                }
                if constexpr (HERE) {
                    unsigned char* const to_row = smem + st * stage_bytes + PR_W_BYTES + (piece >> 2) * half_bytes;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int n = r * 16 + (t >> 3), c = (piece & 3) * 2;
                        if (n >= p.n) break;
                        uint32_t h[8];
                        halves_of(codes[r].x, h[0], h[1]), halves_of(codes[r].y, h[2], h[3]);
                        halves_of(codes[r].z, h[4], h[5]), halves_of(codes[r].w, h[6], h[7]);
                        *reinterpret_cast<uint4*>(to_row + n * 128 + ((c ^ (n & 7)) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4*>(to_row + n * 128 + (((c + 1) ^ (n & 7)) * 16)) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                    specv::fence_proxy_async_shared();
                    fetch(k_from + (k - k_from + 2) % (k_to - k_from));
                }
                const unsigned char* const src = smem + st * stage_bytes + row * 128;
                uint4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const uint4*>(src + ((j ^ (row & 7)) * 16));
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    // the buffer's half is free when the products of step g - 2 have read it; of the second half that is when they are done
                    if (g >= 2) half ? wait(&s_empty[used], used_round & 1) : wait(&s_half_empty[mine], ((g >> 1) - 1) & 1);
                    specc::tmem_fence_after();
#pragma unroll
                    for (int j = 4 * half; j < 4 * half + 4; j += 2) {
                        uint32_t h[16];
                        halves_of(v[j].x, h[0], h[1]), halves_of(v[j].y, h[2], h[3]);
                        halves_of(v[j].z, h[4], h[5]), halves_of(v[j].w, h[6], h[7]);
                        halves_of(v[j + 1].x, h[8], h[9]), halves_of(v[j + 1].y, h[10], h[11]);
                        halves_of(v[j + 1].z, h[12], h[13]), halves_of(v[j + 1].w, h[14], h[15]);
                        specc::tmem_st16(to + 8 * j, h);
                    }
                    specc::tmem_wait_st();
                    specc::tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_first<PAIR>(&s_ready[2 * mine + half]);
                }
                used = st, used_round = round;
            }
        if (used >= 0) wait(&s_half_empty[mine], ((g - 1 - ((g - 1) & 1 ^ mine)) >> 1) & 1);      // no arrival comes in behind the CTA's end
    } else {
        // ================ sums, and the output
        set_registers<136, true>();
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const uint32_t from = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const int in_tile = (warp & 3) * 32 + lane;
        const int low = (warp - 12) >> 2 ? (p.n / 2 + 15) / 16 * 16 : 0, high = (warp - 12) >> 2 ? p.n : (p.n / 2 + 15) / 16 * 16;
        auto look_up = [&](int i, int to) {      // the scales and the places of a tile's tokens
            if (i >= units) return;
            const Unit u(p, i);
            for (int j = tid - 384; j < p.n && u.tile * p.n + j < p.tokens; j += 256) {
                const int t = u.tile * p.n + j, b = t / p.N;
                s_scales[to][j] = p.a_scale[t];
                s_rows[to][j] = b * p.out.sb + (t - b * p.N) * p.out.sn;
            }
            __syncwarp();
        };
        look_up(first, 0);
        int chunk = 0, turn = 0;
        for (int i = first; i < units; i += by, turn ^= 1) {
            const Unit u(p, i);
            const int t0 = u.tile * p.n, nt = min(p.n, p.tokens - t0), mine = min(high, nt) - low;      // tokens; this warp's
            const float* const s_scale = s_scales[turn];
            const long long* const s_row = s_rows[turn];
            __syncwarp();      // this barrier is for whole warps
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const int c = (u.channel * CTAS + (PAIR ? rank : 0)) * PR_CH + in_tile;
            const float ws = c < p.C ? p.w_scale[c] : 0.f, bias = p.bias && c < p.C ? p.bias[c] : 0.f;
            int acc[PR_TOKENS / 2];
#pragma unroll
            for (int j = 0; j < PR_TOKENS / 2; ++j) acc[j] = 0;
            const int chunks = (k_to - k_from + PR_CHUNK - 1) / PR_CHUNK;
            for (int q = 0; q < chunks; ++q, ++chunk) {
                if (q == min(2, chunks - 1)) look_up(i + by, turn ^ 1);      // where there is time
                wait(&s_acc_full[chunk & 1], (chunk >> 1) & 1);
                specc::tmem_fence_after();
#pragma unroll
                for (int j = 0; j < PR_TOKENS / 2; j += 16)
                    if (low + j < high) {
                        uint32_t v[16];
                        specc::tmem_ld(from + (chunk & 1) * PR_TOKENS + low + j, v);
                        if (low + j + 16 >= high) {      // the last of them are out of the accumulator
                            specc::tmem_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive_first<PAIR>(&s_acc_empty[chunk & 1]);
                            __syncwarp();
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[j + e] += __float2int_rn(__uint_as_float(v[e]));
                    }
                if (low >= high && lane == 0) arrive_first<PAIR>(&s_acc_empty[chunk & 1]);      // a narrow tile's other half
            }
            T* const out = static_cast<T*>(p.out.p) + c;
            auto scaled = [&](int j, int sum) {
                return from_float<T>(scaled_sum(sum, s_scale[j] * ws, p.bias != nullptr, bias));
            };
            if (!PAIR && p.split > 1) {
                // one tile a cluster: its CTAs add their sums, each for every split-th token
                int* const part = reinterpret_cast<int*>(smem) + in_tile;
#pragma unroll
                for (int j = 0; j < PR_TOKENS / 2; j += 16)
                    if (j < mine) {
#pragma unroll
                        for (int e = j; e < j + 16; ++e)
                            if (e < mine) part[(low + e) * PR_CH] = acc[e];
                    }
                __syncwarp();
                specv::cluster_sync_all();
                for (int j = rank + ((warp - 12) >> 2) * p.split; j < nt; j += 2 * p.split) {
                    int sum = 0;
                    for (int r = 0; r < p.split; ++r)
                        sum += __float_as_int(specv::ld_cluster_f32(specv::map_to_rank(smem_addr(part + j * PR_CH), r)));
                    const T y = scaled(j, sum);
                    if (c < p.C) out[s_row[j]] = y;
                }
                __syncwarp();
                specv::cluster_sync_all();
            } else {
                // sixteen tokens at a time, their values before their stores, which need not wait for one another
#pragma unroll
                for (int j = 0; j < PR_TOKENS / 2; j += 16)
                    if (j < mine) {
                        T y[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] = scaled(low + j + e, acc[j + e]);
                        if (j + 16 <= mine && c < p.C) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) out[s_row[low + j + e]] = y[e];
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (j + e < mine && c < p.C) out[s_row[low + j + e]] = y[e];
                        }
                    }
            }
        }
    }
    // What follows is run by warps with 48 and with 136 registers: it needs a few.
    __syncwarp();
    if (!PAIR && p.split > 1 && warp < 12) {      // the barriers around the sums' exchange above
        specv::cluster_sync_all();
        specv::cluster_sync_all();
    }
    specc::tmem_fence_before();
    __syncthreads();
    if (PAIR) specv::cluster_sync_all();
    if (warp == 2) {
        specc::tmem_fence_after();
        if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
        else specc::tmem_dealloc(tmem, 512);
    }
}

}  // namespace specs
