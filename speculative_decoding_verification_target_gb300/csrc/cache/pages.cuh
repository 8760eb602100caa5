// Bookkeeping of the cache's pages: fork, reserve, commit, release and compact, all on the device.
#pragma once
#include "cache_format.cuh"

namespace specc {

struct PagesParams {
    unsigned char* pool;
    int* table;
    int* lengths;
    int* refs;
    const int *a, *b;        // src and dst, n_new, advance or slots
    int* out;                // served or used
    int* scratch;            // after the workspace's header
    unsigned* status;
    long long page_bytes;
    int layers, S, M, P, n, extra, window, sinks;
};

constexpr int PG_CLUSTER = 8;            // CTAs of the cluster that reserves or compacts, at most
constexpr int PG_THREADS = 1024;
constexpr int COPY_THREADS = 256;
constexpr int COPY_BYTES = COPY_THREADS * 16 * 4;   // what a CTA copies at a time, four vectors a thread

__device__ __forceinline__ int clamp_length(int len, int M, unsigned* status) {
    const int room = static_cast<int>(min(static_cast<long long>(M) * PAGE, 2147483647LL));
    if (len < 0 || len > room) atomicOr(status, SPEC_STATUS_BAD_LENGTH);
    return min(max(len, 0), room);
}

// Lets go of one table entry: exchanged for -1, so that of two threads on the same entry one counts it down.
__device__ __forceinline__ void drop_entry(const PagesParams& p, int* e) {
    const int page = atomicExch(e, -1);
    if (page < 0) return;
    if (page < p.P) atomicSub(&p.refs[page], 1);
    else atomicOr(p.status, SPEC_STATUS_BAD_PAGE);
}

// One CTA per pair. A destination is never a source of the call (such pairs are left out), so no CTA reads a row
// that another one writes.
__global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ PagesParams p) {
    after_previous();
    const int f = blockIdx.x, src = p.a[f], dst = p.b[f];
    bool bad = src < 0 || src >= p.S || dst < 0 || dst >= p.S;
    for (int i = threadIdx.x; i < p.n; i += blockDim.x) bad |= p.a[i] == dst || (i < f && p.b[i] == dst);
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicOr(p.status, SPEC_STATUS_BAD_SLOT);
        return;
    }
    const int* const from = p.table + static_cast<size_t>(src) * p.M;
    int* const to = p.table + static_cast<size_t>(dst) * p.M;
    for (int j = threadIdx.x; j < p.M; j += blockDim.x) {
        const int page = from[j], old = to[j];
        if (page >= 0 && page < p.P) atomicAdd(&p.refs[page], 1);
        if (old >= 0 && old < p.P) atomicSub(&p.refs[old], 1);
        if (page >= p.P || old >= p.P) atomicOr(p.status, SPEC_STATUS_BAD_PAGE);
        to[j] = page < p.P ? max(page, -1) : -1;
    }
    if (threadIdx.x == 0) p.lengths[dst] = p.lengths[src];
}

// One CTA per sequence: its new length, then the entries past it and those before every later query's window.
__global__ void __launch_bounds__(128) commit_kernel(const __grid_constant__ PagesParams p) {
    after_previous();
    const int s = blockIdx.x;
    __shared__ int s_len;
    if (threadIdx.x == 0) {
        const long long raw = static_cast<long long>(p.lengths[s]) + p.a[s] + p.extra;
        const int len = clamp_length(static_cast<int>(max(min(raw, 2147483647LL), -1LL)), p.M, p.status);
        p.lengths[s] = len;
        s_len = len;
    }
    __syncthreads();
    const long long len = s_len;
    int* const row = p.table + static_cast<size_t>(s) * p.M;
    for (int j = threadIdx.x; j < p.M; j += blockDim.x) {
        const long long lo = static_cast<long long>(j) * PAGE, hi = lo + PAGE;
        const bool gone = lo >= len || (p.window > 0 && lo >= p.sinks && hi <= len - p.window + 1);
        if (gone && row[j] >= 0) drop_entry(p, row + j);
    }
}

__global__ void __launch_bounds__(128) release_kernel(const __grid_constant__ PagesParams p) {
    after_previous();
    const int s = p.a[blockIdx.x];
    if (s < 0 || s >= p.S) {
        if (threadIdx.x == 0) atomicOr(p.status, SPEC_STATUS_BAD_SLOT);
        return;
    }
    int* const row = p.table + static_cast<size_t>(s) * p.M;
    for (int j = threadIdx.x; j < p.M; j += blockDim.x)
        if (row[j] >= 0) drop_entry(p, row + j);
    if (threadIdx.x == 0) p.lengths[s] = 0;
}

// Exclusive sum over the cluster's threads, in order of (CTA, thread), and their total. Every thread of the cluster calls it.
struct ClusterScan {
    unsigned long long warp[32];
    unsigned long long cta;      // this CTA's total, read by the others
};
__device__ __forceinline__ unsigned long long cluster_scan(ClusterScan* sh, unsigned long long v, unsigned rank,
                                                           unsigned long long* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    unsigned long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sh->warp[w] = x;
    __syncthreads();
    if (w == 0) {
        unsigned long long t = sh->warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        sh->warp[lane] = t;
        if (lane == 31) sh->cta = t;
    }
    __syncthreads();
    specv::cluster_sync_all();
    unsigned long long before = 0, all = 0;
    for (unsigned r = 0; r < specv::cluster_nctarank(); ++r) {
        const uint32_t a = specv::map_to_rank(specv::smem_addr(&sh->cta), r);
        unsigned long long t;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(t) : "r"(a) : "memory");
        all += t;
        if (r < rank) before += t;
    }
    const unsigned long long mine = before + (w ? sh->warp[w - 1] : 0ull) + x - v;
    specv::cluster_sync_all();   // nobody overwrites a total that another CTA still reads
    *total = all;
    return mine;
}

// A thread's run of pages: neighbouring ones, so that an exclusive sum over threads is one over page numbers.
struct Run {
    int lo, hi;
};
__device__ __forceinline__ Run run_of(int n, unsigned rank) {
    const long long t = static_cast<long long>(rank) * PG_THREADS + threadIdx.x;
    const long long T = specv::cluster_nctarank() * PG_THREADS;
    return {static_cast<int>(t * n / T), static_cast<int>((t + 1) * n / T)};
}

// What sequence s wants: entries [a, z] of its row, the committed length. False where it wants nothing or cannot
// be served (`fits` false).
struct Want {
    int len, a, z;
    bool fits;
};
__device__ __forceinline__ bool want_of(const PagesParams& p, int s, Want& w) {
    const int n = p.a[s];
    w.fits = true;
    if (n <= 0) return false;
    w.len = p.lengths[s];
    const long long end = static_cast<long long>(w.len) + n;
    w.fits = w.len >= 0 && end <= static_cast<long long>(p.M) * PAGE;
    if (!w.fits) return false;
    w.a = w.len / PAGE;
    w.z = static_cast<int>((end - 1) / PAGE);
    return true;
}
// Whether entry e has to be replaced by a page of the sequence's own: missing, or shared with another sequence.
__device__ __forceinline__ bool wants_page(const PagesParams& p, int e) {
    return e < 0 || e >= p.P || p.refs[e] > 1;
}

// Reservation, by one cluster: counts are exclusive sums over the cluster's threads, so the k-th page wanted and
// the k-th free page meet without sorting and in an order that does not depend on timing. refs stays as the call
// found it until every sequence has read it.
//   scratch: need [S], free list [P], former page [P], copies' source and destination [S] each, then the number of
//   copies and of pages given (the copy kernel reads the first).
__global__ void __launch_bounds__(PG_THREADS) reserve_kernel(const __grid_constant__ PagesParams p) {
    after_previous();
    __shared__ ClusterScan s_scan;
    __shared__ int s_given;
    const unsigned rank = specv::cluster_ctarank();
    const int threads = specv::cluster_nctarank() * PG_THREADS, warps = threads / 32;
    const int lane = threadIdx.x & 31, gw = rank * (PG_THREADS / 32) + (threadIdx.x >> 5);
    int* const need = p.scratch;
    int* const free_list = need + p.S;
    int* const former = free_list + p.P;
    int* const copy_src = former + p.P;
    int* const copy_dst = copy_src + p.S;
    int* const counts = copy_dst + p.S;
    if (rank == 0 && threadIdx.x == 0) counts[0] = counts[1] = 0;
    if (threadIdx.x == 0) s_given = 0;

    // pages wanted by each sequence, a warp to a sequence
    for (int s = gw; s < p.S; s += warps) {
        Want w;
        int c = 0;
        if (want_of(p, s, w)) {
            const int* const row = p.table + static_cast<size_t>(s) * p.M;
            for (int j = w.a + lane; j <= w.z; j += 32) {
                const int e = row[j];
                if (e >= p.P) atomicOr(p.status, SPEC_STATUS_BAD_PAGE);
                c += wants_page(p, e);
            }
            c = __reduce_add_sync(0xffffffffu, c);
        } else if (!w.fits && lane == 0) {
            atomicOr(p.status, SPEC_STATUS_BAD_LENGTH);
        }
        if (lane == 0) need[s] = w.fits ? c : -1;
    }
    // the free pages of each thread's run
    const Run r = run_of(p.P, rank);
    int mine = 0;
#pragma unroll 4
    for (int i = r.lo; i < r.hi; ++i) mine += p.refs[i] <= 0;
    unsigned long long all_free;
    const unsigned long long first_free = cluster_scan(&s_scan, static_cast<unsigned long long>(mine), rank, &all_free);
    {
        unsigned long long k = first_free;
        for (int i = r.lo; i < r.hi; ++i)
            if (p.refs[i] <= 0) free_list[k++] = i;
    }
    // (cluster_scan's barriers made need[] visible) which sequences are served, and where their pages start
    const Run q = run_of(p.S, rank);
    unsigned long long sum = 0, total;
    for (int s = q.lo; s < q.hi; ++s) sum += static_cast<unsigned long long>(max(need[s], 0));
    unsigned long long at = cluster_scan(&s_scan, sum, rank, &total);
    int given = 0;
    for (int s = q.lo; s < q.hi; ++s) {
        const int c = need[s];
        const bool ok = c >= 0 && (c == 0 || at + c <= all_free);
        if (c > 0 && !ok) atomicOr(p.status, SPEC_STATUS_NO_PAGES);
        if (p.out) p.out[s] = ok;
        need[s] = ok && c > 0 ? static_cast<int>(at) : -1;   // from here on: the first of its pages, or none
        at += c > 0 ? c : 0;
        if (ok && c > 0) given = static_cast<int>(at);
    }
    if (given) atomicMax(&s_given, given);
    __syncthreads();
    if (threadIdx.x == 0 && s_given) atomicMax(&counts[1], s_given);
    specv::cluster_sync_all();
    // hand them out
    for (int s = gw; s < p.S; s += warps) {
        int k = need[s];
        Want w;
        if (k < 0 || !want_of(p, s, w)) continue;
        int* const row = p.table + static_cast<size_t>(s) * p.M;
        for (int j0 = w.a; j0 <= w.z; j0 += 32) {
            const int j = j0 + lane;
            const int e = j <= w.z ? row[j] : 0;
            const bool take = j <= w.z && wants_page(p, e);
            const unsigned m = __ballot_sync(0xffffffffu, take);
            if (take) {
                const int kk = k + __popc(m & ((1u << lane) - 1u)), page = free_list[kk];
                const bool held = e >= 0 && e < p.P;
                former[kk] = held ? e : -1;
                row[j] = page;
                if (held && j == w.a && w.len % PAGE) {
                    const int c = atomicAdd(&counts[0], 1);   // any order: the copies are of different pages
                    copy_src[c] = e;
                    copy_dst[c] = page;
                }
            }
            k += __popc(m);
        }
    }
    specv::cluster_sync_all();
    const int n = *static_cast<volatile int*>(&counts[1]);
    for (int k = static_cast<int>(rank) * PG_THREADS + threadIdx.x; k < n; k += threads) {
        p.refs[free_list[k]] = 1;
        if (former[k] >= 0) atomicSub(&p.refs[former[k]], 1);
    }
}

// Copies of whole pages in every layer: page src[i] to dst[i], i < count. Grid-stride over pieces of COPY_BYTES, by 16 CTAs an
// SM: half of a pool of 1.1 GB moved, 570 MB read and written, takes 85 us, 6.7 TB/s, the copy rate (4, 6, 8 and 16 CTAs an SM:
// the whole compaction 101, 109, 101 and 99 us).
__device__ __forceinline__ void copy_pages(const PagesParams& p, const int* src, const int* dst, int count) {
    const long long pieces = (p.page_bytes + COPY_BYTES - 1) / COPY_BYTES;
    const long long work = pieces * count * p.layers;
    for (long long i = blockIdx.x; i < work; i += gridDim.x) {
        const long long q = i / pieces, piece = i - q * pieces;
        const int l = static_cast<int>(q / count), c = static_cast<int>(q - static_cast<long long>(l) * count);
        const long long base = static_cast<long long>(l) * p.P;
        const unsigned char* const from = p.pool + (base + src[c]) * p.page_bytes;
        unsigned char* const to = p.pool + (base + dst[c]) * p.page_bytes;
        const long long o = piece * COPY_BYTES + threadIdx.x * 16;
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (o + k * COPY_THREADS * 16 < p.page_bytes) v[k] = __ldcs(reinterpret_cast<const uint4*>(from + o + k * COPY_THREADS * 16));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (o + k * COPY_THREADS * 16 < p.page_bytes) __stcs(reinterpret_cast<uint4*>(to + o + k * COPY_THREADS * 16), v[k]);
    }
}

__global__ void __launch_bounds__(COPY_THREADS) reserve_copy_kernel(const __grid_constant__ PagesParams p) {
    after_previous();
    const int* const copy_src = p.scratch + p.S + 2 * static_cast<long long>(p.P);
    copy_pages(p, copy_src, copy_src + p.S, copy_src[2 * p.S]);
}

// The moves of a compaction, by one cluster. With n pages in use, movers (used, number >= n) and holes (free, number < n) are
// as many, and the i-th of the one goes to the i-th of the other. One sum serves both: with u used pages before it, a hole i is
// the (i - u)-th, and a mover stands at u of the used pages, of which the movers are the last.
//   scratch: used pages from n on, by rank [P], holes [P], new number of pages n .. P - 1 [P], number of moves, n.
__global__ void __launch_bounds__(PG_THREADS) compact_plan_kernel(const __grid_constant__ PagesParams p) {
    after_previous();
    __shared__ ClusterScan s_scan;
    const unsigned rank = specv::cluster_ctarank();
    const int threads = specv::cluster_nctarank() * PG_THREADS;
    int* const movers = p.scratch;
    int* const holes = movers + p.P;
    int* const remap = holes + p.P;
    int* const counts = remap + p.P;
    const Run r = run_of(p.P, rank);
    unsigned long long used = 0, n64;
#pragma unroll 4
    for (int i = r.lo; i < r.hi; ++i) used += p.refs[i] > 0;
    int u = static_cast<int>(cluster_scan(&s_scan, used, rank, &n64));
    const int n = static_cast<int>(n64);
#pragma unroll 4
    for (int i = r.lo; i < r.hi; ++i) {
        if (i == n) counts[0] = n - u;
        if (p.refs[i] > 0) {
            if (i >= n) movers[u] = i;
            ++u;
        } else if (i < n) {
            holes[i - u] = i;
        } else {
            remap[i - n] = i;
        }
    }
    if (rank == 0 && threadIdx.x == 0) {
        if (n == p.P) counts[0] = 0;
        counts[1] = n;
        if (p.out) p.out[0] = n;
    }
    specv::cluster_sync_all();
    const int moves = *static_cast<volatile int*>(&counts[0]);
    for (int k = static_cast<int>(rank) * PG_THREADS + threadIdx.x; k < moves; k += threads) {
        const int from = movers[n - moves + k], to = holes[k];
        remap[from - n] = to;
        p.refs[to] = p.refs[from];
        p.refs[from] = 0;
    }
}

// The copies and the table's new page numbers. Holes are free and movers are in use, so no copy reads a page that
// another one writes.
__global__ void __launch_bounds__(COPY_THREADS) compact_move_kernel(const __grid_constant__ PagesParams p) {
    after_previous();
    const int* const movers = p.scratch;
    const int* const remap = movers + 2 * static_cast<long long>(p.P);
    const int moves = remap[p.P], n = remap[p.P + 1];
    const long long entries = static_cast<long long>(p.S) * p.M;
    for (long long i = static_cast<long long>(blockIdx.x) * COPY_THREADS + threadIdx.x; i < entries;
         i += static_cast<long long>(gridDim.x) * COPY_THREADS) {
        const int e = p.table[i];
        if (e >= n && e < p.P) p.table[i] = remap[e - n];
        if (e >= p.P) atomicOr(p.status, SPEC_STATUS_BAD_PAGE);
    }
    copy_pages(p, movers + (n - moves), movers + p.P, moves);
}

}  // namespace specc
