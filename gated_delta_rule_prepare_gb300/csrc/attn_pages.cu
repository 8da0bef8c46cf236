// Pages of the 4-bit cache: kda_attn_kv4_resize, _fork and _compact keep the page
// table and the pages' counts on the device, kda_attn_kv4_copy moves pages.
//
// The three are passes over small integer arrays, each pass needing what the last one
// counted: latency is what they take.  One cluster of up to eight CTAs runs all
// passes of a call, two or three of its barriers between them (512 rows of 128 pages, 40000
// pages: fork 18.5 us, compact 13.3, resize 8.1); few entries run in one CTA.  Arrays are cut
// into one slice for each warp; a warp counts what it looks for in its slice, the counts are
// summed up in the order of the slices, and on a second pass each thing found knows its number.
// So new pages come in order, and no result depends on which warp was first: what is added to
// a count atomically is integers.  What is known of rows (fork) each CTA works out by itself.
//
// Arrays that one pass writes and another CTA reads are read through L2 (__ldcg).
#include <cooperative_groups.h>

#include "attn_common.h"

namespace kda {
namespace {

using namespace attn;
namespace cg = cooperative_groups;

__device__ unsigned g_pages_status = 0;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMostCtas = 8;
constexpr int kRowsShared = 12288;  // rows of a fork whose four integers fit shared memory
constexpr int kMostInts = 0x7ff00000;  // of a table, of pages: a grid's step more is an int

struct PageArgs {
    const int *table, *lens, *refs, *parent;
    int *table_out, *lens_out, *refs_out, *src, *dst, *count;
    int n_seqs, width, n_pages, page_shift;
    // workspace
    int* want;          // [n_seqs * width] entries that want a page, in order (resize)
    int* rows;          // [kMostCtas][4 * n_seqs] what a CTA knows of the rows, if they are many
    int* staged_table;  // a copy of the table where the output is in its place
    int* place;         // [n_pages] where each page goes, -1 for free ones

    __device__ __forceinline__ int held(int len) const {
        return (int)(((long long)len + (1 << page_shift) - 1) >> page_shift);
    }
    __device__ __forceinline__ bool names(int v) const { return v >= 0 && v < n_pages; }
    __device__ __forceinline__ int clamped_len(int len, unsigned& bad) const {
        const long long most = (long long)width << page_shift;
        if (len < 0 || len > most) bad |= STATUS_BAD_PAGES;
        return (int)min(max((long long)len, 0LL), most);
    }
};

// One cluster's threads, and sums over its warps.
struct Team {
    cg::cluster_group cluster = cg::this_cluster();
    int rank, ctas, warp, lane, id, threads, me;
    int (*sums)[kWarps];  // [2]: of one sum, and of the next one

    __device__ explicit Team(int (*shared_sums)[kWarps]) : sums(shared_sums) {
        rank = (int)cluster.block_rank();
        ctas = (int)cluster.num_blocks();
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        id = rank * kWarps + warp;
        threads = ctas * kThreads;
        me = rank * kThreads + threadIdx.x;
    }
    __device__ void sync() {
        __threadfence();
        cluster.sync();
    }
    // This warp's part of [0, n), in pieces of 32.
    struct Slice {
        int from, to;
    };
    __device__ Slice slice(int n, int of) const {
        const int warps = ctas * kWarps;
        const int each = (int)(((long long)n + 32LL * warps - 1) / (32LL * warps)) * 32;
        const int from = (int)min((long long)n, (long long)each * of);
        return {from, (int)min((long long)n, from + (long long)each)};
    }
    __device__ Slice slice(int n) const { return slice(n, id); }
    // One number a warp (the same in its lanes): the sum over the warps before this one,
    // and over all.  A barrier of the cluster; `which` alternates between 0 and 1.
    __device__ int before(int x, int which, int& total) {
        if (lane == 0) sums[which][warp] = x;
        sync();
        int mine = 0, all = 0;
        for (int r = 0; r < ctas; ++r) {
            const int y = cluster.map_shared_rank(&sums[which][0], r)[lane];
            const int s = __reduce_add_sync(0xffffffffu, y);
            if (r < rank) mine += s;
            if (r == rank) mine += __reduce_add_sync(0xffffffffu, lane < warp ? y : 0);
            all += s;
        }
        total = all;
        return mine;
    }
    // Before a CTA ends: others may still read its sums.
    __device__ void leave(unsigned bad) {
        if (bad) atomicOr(&g_pages_status, bad);
        cluster.sync();
    }
};

// How many pages of a warp's slice are free, and each of them with its number.
constexpr int kAhead = 4;  // steps of 32 pages loaded at a time
__device__ __forceinline__ int count_free(const Team& t, const PageArgs& a) {
    const Team::Slice s = t.slice(a.n_pages);
    int mine = 0;
    for (int i0 = s.from; i0 < s.to; i0 += 32 * kAhead) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + 32 * k + t.lane;
            mine += i < s.to && __ldcg(a.refs_out + i) <= 0;
        }
    }
    return __reduce_add_sync(0xffffffffu, mine);
}
template <class Take>
__device__ __forceinline__ void take_free(const Team& t, const PageArgs& a, int at, int wanted,
                                          Take take) {
    const Team::Slice s = t.slice(a.n_pages);
    for (int i0 = s.from; i0 < s.to && at < wanted; i0 += 32) {
        const int i = i0 + t.lane;
        const bool free = i < s.to && __ldcg(a.refs_out + i) <= 0;
        const unsigned all = __ballot_sync(0xffffffffu, free);
        const int n = at + __popc(all & ((1u << t.lane) - 1));
        if (free && n < wanted) {
            a.refs_out[i] = 1;
            take(n, i);
        }
        at += __popc(all);
    }
}

__global__ void __launch_bounds__(kThreads) resize_kernel(PageArgs a) {
    __shared__ int sums[2][kWarps];
    Team t(sums);
    pdl_wait();
    pdl_release();
    unsigned bad = 0;
    const Team::Slice s = t.slice(a.n_seqs * a.width);
    // Entries past a sequence's length give their pages up; missing ones are counted, and
    // the steps that have some noted (as far as the mask goes).
    int mine = 0;
    unsigned long long steps = 0;
    auto missing = [&](int i, int v) {
        unsigned ignore = 0;
        const int n = i / a.width, col = i - n * a.width;
        return col < a.held(a.clamped_len(__ldcg(a.lens + n), ignore)) && !a.names(v);
    };
    for (int i0 = s.from; i0 < s.to; i0 += 32 * kAhead) {
        int v[kAhead], len[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + 32 * k + t.lane;
            if (i < s.to) v[k] = a.table_out[i], len[k] = __ldcg(a.lens + i / a.width);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + 32 * k + t.lane;
            bool miss = false;
            if (i < s.to) {
                if (v[k] < -1 || v[k] >= a.n_pages) bad |= STATUS_BAD_PAGES;
                const bool wanted = i % a.width < a.held(a.clamped_len(len[k], bad));
                const bool there = a.names(v[k]);
                miss = wanted && !there;
                if (!wanted && there) atomicAdd(a.refs_out + v[k], -1);
                if (v[k] != -1 && !(wanted && there)) a.table_out[i] = -1;
            }
            const unsigned found = __ballot_sync(0xffffffffu, miss);
            mine += __popc(found);
            if (found) steps |= 1ull << min((i0 - s.from) / 32 + k, 63);
        }
    }
    int wanted, at = t.before(mine, 0, wanted);
    if (wanted) {
        if (mine) {  // the entries in order
            for (int i0 = s.from; i0 < s.to; i0 += 32) {
                if (!(steps >> min((i0 - s.from) / 32, 63) & 1)) continue;
                const int i = i0 + t.lane;
                const bool miss = i < s.to && missing(i, a.table_out[i]);
                const unsigned all = __ballot_sync(0xffffffffu, miss);
                if (miss) a.want[at + __popc(all & ((1u << t.lane) - 1))] = i;
                at += __popc(all);
            }
        }
        int there;
        const int first = t.before(count_free(t, a), 1, there);
        take_free(t, a, first, wanted,
                  [&](int n, int page) { a.table_out[__ldcg(a.want + n)] = page; });
        if (there < wanted) bad |= STATUS_NO_PAGES;
    }
    t.leave(bad);
}

// What a CTA knows of a fork's rows: each one's parent (-1: none) and its length, each
// parent's lowest child, and the rows that get a page of their own, in order.
struct ForkRows {
    int *parent, *len, *first, *copies;
};

__global__ void __launch_bounds__(kThreads) fork_kernel(PageArgs a) {
    extern __shared__ int row_memory[];
    __shared__ int sums[2][kWarps], scan[kWarps];
    Team t(sums);
    pdl_wait();
    pdl_release();
    unsigned bad = 0;
    const int n_seqs = a.n_seqs, tid = threadIdx.x, entries = n_seqs * a.width;
    int* const rows = n_seqs <= kRowsShared ? row_memory : a.rows + (size_t)t.rank * 4 * n_seqs;
    const ForkRows r = {rows, rows + n_seqs, rows + 2 * n_seqs, rows + 3 * n_seqs};
    const int* table = a.table;
    if (a.table == a.table_out) {
        for (int i = t.me; i < entries; i += t.threads) a.staged_table[i] = __ldcg(a.table + i);
        table = a.staged_table;
    }
    if (a.refs != a.refs_out)
        for (int i = t.me; i < a.n_pages; i += t.threads) a.refs_out[i] = __ldcg(a.refs + i);
    for (int n = tid; n < n_seqs; n += kThreads) {
        const int p = __ldcg(a.parent + n);
        if (p < -1 || p >= n_seqs) bad |= STATUS_BAD_PAGES;
        const bool live = p >= 0 && p < n_seqs;
        r.parent[n] = live ? p : -1;
        r.len[n] = live ? a.clamped_len(__ldcg(a.lens + p), bad) : 0;
        r.first[n] = n_seqs;
    }
    // (everybody has read lens, which lens_out may be)
    t.sync();
    for (int n = tid; n < n_seqs; n += kThreads)
        if (r.parent[n] >= 0) atomicMin(r.first + r.parent[n], n);
    __syncthreads();
    auto copied = [&](int n) {
        return r.parent[n] >= 0 && (r.len[n] & ((1 << a.page_shift) - 1)) &&
               r.first[r.parent[n]] != n;
    };
    // the table, less the pages to come, and what that changes in the counts
    for (int i0 = t.me; i0 < entries; i0 += kAhead * t.threads) {
        int old[kAhead], now[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * t.threads;
            old[k] = now[k] = -1;
            if (i >= entries) continue;
            const int n = i / a.width, col = i - n * a.width;
            old[k] = __ldcg(table + i);
            if (col < a.held(r.len[n]) - (copied(n) ? 1 : 0))
                now[k] = __ldcg(table + r.parent[n] * a.width + col);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * t.threads;
            if (i >= entries) continue;
            if (old[k] < -1 || old[k] >= a.n_pages) bad |= STATUS_BAD_PAGES;
            if (!a.names(now[k])) now[k] = -1;
            if (old[k] != now[k]) {
                if (a.names(old[k])) atomicAdd(a.refs_out + old[k], -1);
                if (now[k] >= 0) atomicAdd(a.refs_out + now[k], 1);
            }
            a.table_out[i] = now[k];
        }
    }
    // the rows that get a page, in order
    int wanted = 0;
    for (int n0 = 0; n0 < n_seqs; n0 += kThreads) {
        const int n = n0 + tid;
        const bool copy = n < n_seqs && copied(n);
        const unsigned all = __ballot_sync(0xffffffffu, copy);
        if (t.lane == 0) scan[t.warp] = __popc(all);
        __syncthreads();
        const int y = scan[t.lane];
        const int at = wanted + __reduce_add_sync(0xffffffffu, t.lane < t.warp ? y : 0);
        wanted += __reduce_add_sync(0xffffffffu, y);
        if (copy) r.copies[at + __popc(all & ((1u << t.lane) - 1))] = n;
        __syncthreads();
    }
    t.sync();  // the counts are complete
    int there = 0;
    if (wanted) {
        const int first = t.before(count_free(t, a), 0, there);
        there = min(there, wanted);
        take_free(t, a, first, wanted, [&](int k, int page) {
            const int n = r.copies[k], last = a.held(r.len[n]) - 1;
            a.table_out[n * a.width + last] = page;
            a.src[k] = __ldcg(table + r.parent[n] * a.width + last);
            a.dst[k] = page;
        });
        if (there < wanted) bad |= STATUS_NO_PAGES;
    }
    for (int n = t.me; n < n_seqs; n += t.threads) {
        if (n >= there) a.src[n] = a.dst[n] = -1;
        a.lens_out[n] = r.len[n];
    }
    __syncthreads();
    // rows that got no page keep their parents' full ones
    for (int k = there + tid; k < wanted; k += kThreads) {
        const int n = r.copies[k];
        if (n % t.threads / kThreads == t.rank)
            a.lens_out[n] = r.len[n] >> a.page_shift << a.page_shift;
    }
    if (t.me == 0) a.count[0] = there;
    t.leave(bad);
}

__global__ void __launch_bounds__(kThreads) compact_kernel(PageArgs a) {
    __shared__ int sums[2][kWarps], high;
    Team t(sums);
    pdl_wait();
    pdl_release();
    unsigned bad = 0;
    const Team::Slice s = t.slice(a.n_pages);
    int mine = 0;
    for (int i0 = s.from; i0 < s.to; i0 += 32 * kAhead) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + 32 * k + t.lane;
            mine += i < s.to && __ldcg(a.refs + i) > 0;
        }
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    int used, at = t.before(mine, 0, used);
    // How many pages move: those in use from `used` on.  Whole slices behind it, and the
    // rest of its own one (each CTA for itself).
    if (t.warp == 0) {
        int count = 0, own = -1;
        for (int of = t.lane; of < t.ctas * kWarps; of += 32) {
            const Team::Slice x = t.slice(a.n_pages, of);
            if (x.from >= used)
                count += t.cluster.map_shared_rank(&sums[0][0], of / kWarps)[of % kWarps];
            else if (x.to > used)
                own = of;
        }
        own = __reduce_max_sync(0xffffffffu, own);
        if (own >= 0) {
            const Team::Slice x = t.slice(a.n_pages, own);
            for (int i = used + t.lane; i < x.to; i += 32) count += __ldcg(a.refs + i) > 0;
        }
        count = __reduce_add_sync(0xffffffffu, count);
        if (t.lane == 0) high = count;
    }
    __syncthreads();
    const int moved = high, low = used - moved;  // pages in use that stay
    for (int i0 = s.from; i0 < s.to; i0 += 32) {
        const int i = i0 + t.lane;
        const int count = i < s.to ? __ldcg(a.refs + i) : 0;
        const unsigned all = __ballot_sync(0xffffffffu, count > 0);
        const int below = at + __popc(all & ((1u << t.lane) - 1));  // pages in use before i
        at += __popc(all);
        if (i >= s.to) continue;
        a.place[i] = count > 0 ? i : -1;
        if (i < used && count <= 0) a.dst[i - below] = i;
        if (i >= used && count > 0) a.src[below - low] = i;
        if (a.refs != a.refs_out) a.refs_out[i] = count;
    }
    for (int k = moved + t.me; k < a.n_pages / 2; k += t.threads) a.src[k] = a.dst[k] = -1;
    t.sync();
    for (int k = t.me; k < moved; k += t.threads) {
        const int from = __ldcg(a.src + k), to = __ldcg(a.dst + k);
        const int count = __ldcg(a.refs + from);
        a.refs_out[to] = count;
        a.refs_out[from] = 0;
        a.place[from] = to;
    }
    t.sync();
    const int entries = a.n_seqs * a.width;
    for (int i0 = t.me; i0 < entries; i0 += kAhead * t.threads) {
        int v[kAhead], now[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * t.threads;
            v[k] = i < entries ? __ldcg(a.table + i) : -1;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) now[k] = a.names(v[k]) ? __ldcg(a.place + v[k]) : -1;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * t.threads;
            if (i >= entries) continue;
            // (an entry whose page is free by its count names none)
            if (v[k] != -1 && now[k] < 0) bad |= STATUS_BAD_PAGES;
            a.table_out[i] = now[k];
        }
    }
    if (t.me == 0) a.count[0] = moved;
    t.leave(bad);
}

// Pages move in equal pieces of at most 32 KB, a CTA each, eight 16-byte loads a thread in flight;
// twice the CTAs that fit, so that those that start behind others even them out: 1.06 GB in and
// out in 160 us, 6.6 TB/s (pieces of 16 KB, CTAs that fit: 12 us more).
constexpr int kCopyThreads = 256;
constexpr int kPiece = 32768;
struct Caches {
    uint8_t* at[KDA_KV4_MAX_CACHES];
};
__global__ void __launch_bounds__(kCopyThreads)
copy_kernel(const __grid_constant__ Caches caches, int n_caches, long long n_pages,
            long long page_bytes, const int* src, const int* dst, const int* count, int most) {
    pdl_wait();
    pdl_release();
    const int pairs = min(max(__ldcg(count), 0), most);
    const long long pieces = (page_bytes + kPiece - 1) / kPiece;
    const long long each = (page_bytes / 16 + pieces - 1) / pieces;  // 16 bytes, of a piece
    const long long total = (long long)pairs * n_caches * pieces;
    for (long long i = blockIdx.x; i < total; i += gridDim.x) {
        const long long page = i / pieces, pair = page / n_caches;
        const int s = __ldcg(src + pair), d = __ldcg(dst + pair);
        if (s < 0 || s >= n_pages || d < 0 || d >= n_pages) {
            if (threadIdx.x == 0) atomicOr(&g_pages_status, STATUS_BAD_PAGES);
            continue;
        }
        uint8_t* cache = caches.at[page - pair * n_caches];
        const long long from = (i - page * pieces) * each;
        const int n = (int)min(each, page_bytes / 16 - from);
        const uint4* x = reinterpret_cast<const uint4*>(cache + s * page_bytes) + from;
        uint4* y = reinterpret_cast<uint4*>(cache + d * page_bytes) + from;
        constexpr int kLoads = kPiece / 16 / kCopyThreads;
        uint4 u[kLoads];
#pragma unroll
        for (int e = 0; e < kLoads; ++e)
            if ((int)threadIdx.x + e * kCopyThreads < n)
                u[e] = __ldcs(x + threadIdx.x + e * kCopyThreads);
#pragma unroll
        for (int e = 0; e < kLoads; ++e)
            if ((int)threadIdx.x + e * kCopyThreads < n)
                __stcs(y + threadIdx.x + e * kCopyThreads, u[e]);
    }
}

struct Layout {
    size_t want, rows, table, place, bytes;
};
Layout workspace_layout(long long n_pages, long long n_seqs, long long width) {
    auto round = [](long long ints) { return (size_t)((ints * 4 + 15) / 16 * 16); };
    Layout l;
    l.want = 0;  // (a table is staged by fork, its missing entries listed by resize)
    l.table = 0;
    l.rows = l.table + round(n_seqs * width);
    l.place = l.rows + (n_seqs > kRowsShared ? round(kMostCtas * 4 * n_seqs) : 0);
    l.bytes = l.place + round(n_pages);
    return l;
}

bool int_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

kda_status pages_call(const char* fn, void (*kernel)(PageArgs), PageArgs a, int64_t n_pages,
                      int page, void* workspace, size_t workspace_bytes, uint64_t stream) {
    KDA_REQUIRE(page == 16 || page == 32 || page == 64 || page == 128 || page == 256,
                KDA_ERR_UNSUPPORTED, "%s: pages of %d tokens (only 16, 32, 64, 128, 256)", fn,
                page);
    KDA_REQUIRE(a.n_seqs >= 1 && a.width >= 1 && a.width <= 0x7fffffff / page && n_pages >= 1 &&
                    n_pages < kMostInts,
                KDA_ERR_INVALID_ARG,
                "%s: n_seqs (%d), max_pages (%d) and n_pages (%lld) must be positive, max_pages "
                "* page below 2^31, n_pages below 2^31 - 2^20",
                fn, a.n_seqs, a.width, (long long)n_pages);
    KDA_REQUIRE((long long)a.n_seqs * a.width < kMostInts, KDA_ERR_INVALID_ARG,
                "%s: a page table of 2^31 - 2^20 entries or more", fn);
    const void* all[] = {a.table, a.table_out, a.refs, a.refs_out};
    for (const void* p : all)
        KDA_REQUIRE(p && int_aligned(p), KDA_ERR_INVALID_ARG,
                    "%s: a null pointer argument, or one that is not 4-byte aligned", fn);
    const void* some[] = {a.lens, a.parent, a.lens_out, a.src, a.dst, a.count};
    for (const void* p : some)
        KDA_REQUIRE(int_aligned(p), KDA_ERR_INVALID_ARG, "%s: an array is not 4-byte aligned", fn);
    const Layout l = workspace_layout(n_pages, a.n_seqs, a.width);
    KDA_REQUIRE(workspace && workspace_bytes >= l.bytes, KDA_ERR_WORKSPACE,
                "%s: workspace of %zu B, %zu B needed", fn, workspace ? workspace_bytes : 0,
                l.bytes);
    KDA_REQUIRE(aligned16(workspace), KDA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned",
                fn);
    KDA_REQUIRE(!fault_injected(), KDA_ERR_CUDA, "%s: injected launch failure", fn);
    a.n_pages = (int)n_pages;
    a.page_shift = __builtin_ctz((unsigned)page);
    char* ws = static_cast<char*>(workspace);
    a.want = reinterpret_cast<int*>(ws + l.want);
    a.rows = reinterpret_cast<int*>(ws + l.rows);
    a.staged_table = reinterpret_cast<int*>(ws + l.table);
    a.place = reinterpret_cast<int*>(ws + l.place);
    // more CTAs wait less for memory and longer for one another (fork of 33 rows, 2160 integers:
    // 1, 4 and 8 take 7.3, 7.7 and 8.4 us; of 64 rows, 7096: 11.1, 8.2 and 8.9; of 512 rows,
    // 32384: 29.0, 13.2 and 10.7)
    const long long ints = n_pages + (long long)a.n_seqs * a.width;
    const int ctas = ints <= 3000 ? 1 : ints <= 12000 ? 4 : kMostCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = as_stream(stream);
    if (kernel == fork_kernel && a.n_seqs <= kRowsShared) {
        cfg.dynamicSmemBytes = 16 * (size_t)a.n_seqs;
        const cudaError_t e =
            cfg.dynamicSmemBytes <= 48 * 1024 - 1024
                ? cudaSuccess
                : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       16 * kRowsShared);
        KDA_REQUIRE(e == cudaSuccess, KDA_ERR_CUDA, "%s: cannot reserve shared memory: %s", fn,
                    cudaGetErrorString(e));
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaLaunchKernelEx(&cfg, kernel, a);
    return launch_result(fn);
}

}  // namespace

cudaError_t status_word_pages(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_pages_status);
}

}  // namespace kda

using namespace kda;

extern "C" size_t kda_attn_kv4_pages_workspace_size(int64_t n_pages, int n_seqs, int max_pages) {
    if (n_pages < 1 || n_pages >= kMostInts || n_seqs < 1 || max_pages < 1 ||
        (long long)n_seqs * max_pages >= kMostInts)
        return 0;
    return workspace_layout(n_pages, n_seqs, max_pages).bytes;
}

extern "C" kda_status kda_attn_kv4_resize(int* page_table, const int* lens, int* refs, int n_seqs,
                                          int max_pages, int64_t n_pages, int page,
                                          void* workspace, size_t workspace_bytes,
                                          uint64_t stream) {
    const char* fn = "kda_attn_kv4_resize";
    PageArgs a = {};
    a.table = a.table_out = page_table;
    a.lens = lens;
    a.refs = a.refs_out = refs;
    a.n_seqs = n_seqs, a.width = max_pages;
    KDA_REQUIRE(lens, KDA_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    return pages_call(fn, resize_kernel, a, n_pages, page, workspace, workspace_bytes, stream);
}

extern "C" kda_status kda_attn_kv4_fork(const int* page_table, const int* lens, const int* refs,
                                        const int* parent, int* page_table_out, int* lens_out,
                                        int* refs_out, int* src, int* dst, int* count, int n_seqs,
                                        int max_pages, int64_t n_pages, int page, void* workspace,
                                        size_t workspace_bytes, uint64_t stream) {
    const char* fn = "kda_attn_kv4_fork";
    const PageArgs a = {page_table, lens, refs, parent, page_table_out, lens_out, refs_out,
                        src, dst, count, n_seqs, max_pages};
    KDA_REQUIRE(lens && parent && lens_out && src && dst && count, KDA_ERR_INVALID_ARG,
                "%s: null pointer argument", fn);
    return pages_call(fn, fork_kernel, a, n_pages, page, workspace, workspace_bytes, stream);
}

extern "C" kda_status kda_attn_kv4_compact(const int* page_table, const int* refs,
                                           int* page_table_out, int* refs_out, int* src, int* dst,
                                           int* count, int n_seqs, int max_pages, int64_t n_pages,
                                           void* workspace, size_t workspace_bytes,
                                           uint64_t stream) {
    const char* fn = "kda_attn_kv4_compact";
    const PageArgs a = {page_table, nullptr, refs, nullptr, page_table_out, nullptr, refs_out,
                        src, dst, count, n_seqs, max_pages};
    KDA_REQUIRE((n_pages < 2 || (src && dst)) && count, KDA_ERR_INVALID_ARG,
                "%s: null pointer argument", fn);
    return pages_call(fn, compact_kernel, a, n_pages, 16, workspace, workspace_bytes, stream);
}

extern "C" kda_status kda_attn_kv4_copy(uint8_t* const* caches, int n_caches, int64_t n_pages,
                                        int page, int kv_heads, const int* src, const int* dst,
                                        const int* count, int max_count, uint64_t stream) {
    const char* fn = "kda_attn_kv4_copy";
    KDA_REQUIRE(n_caches >= 1 && n_caches <= KDA_KV4_MAX_CACHES && caches, KDA_ERR_INVALID_ARG,
                "%s: n_caches (%d) must be 1 to %d, and caches an array of them", fn, n_caches,
                KDA_KV4_MAX_CACHES);
    KDA_REQUIRE(max_count >= 0, KDA_ERR_INVALID_ARG, "%s: max_count (%d) must be >= 0", fn,
                max_count);
    if (max_count == 0) return KDA_OK;
    Caches c = {};
    for (int i = 0; i < n_caches; ++i) {
        const kda_status st = validate_cache(fn, caches[i], n_pages, page, src, 1, dst, 1,
                                             kv_heads, D);
        if (st != KDA_OK) return st;
        c.at[i] = caches[i];
    }
    KDA_REQUIRE(count && int_aligned(count), KDA_ERR_INVALID_ARG,
                "%s: count must be 4-byte aligned and not null", fn);
    KDA_REQUIRE(!fault_injected(), KDA_ERR_CUDA, "%s: injected launch failure", fn);
    const long long bytes = (long long)page * kv_heads * kTokenBytes;
    const long long most = (bytes + kPiece - 1) / kPiece * n_caches * max_count;
    const unsigned grid = (unsigned)(most < 152 * 16 ? most : 152 * 16);
    launch_pdl(copy_kernel, dim3(grid), dim3(kCopyThreads), 0, as_stream(stream), c, n_caches,
               (long long)n_pages, bytes, src, dst, count, max_count);
    return launch_result(fn);
}
