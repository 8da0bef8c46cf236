// Pages of the 4-bit cache: kda_attn_kv4_resize, _fork and _compact keep the page
// table and the pages' counts on the device, kda_attn_kv4_copy moves pages.
//
// The three are passes over small integer arrays, each pass needing what the last one
// counted: latency is what they take.  One cluster of up to eight CTAs runs all
// passes of a call, with its barrier between them; few entries run in one CTA.
// An array is cut into one slice for each warp; a warp counts what it looks for in
// its slice, the counts are summed up in the order of the slices, and on a second
// pass each thing found knows its number.  So new pages come in order, and no result
// depends on which warp was first: what is added to a count atomically is integers.
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

struct PageArgs {
    const int *table, *lens, *refs, *parent;
    int *table_out, *lens_out, *refs_out, *src, *dst, *count;
    int n_seqs, width, n_pages, page_shift;
    // workspace
    int* got;    // [n_seqs * width at most] new pages, in order (resize: entries, fork: rows)
    int* first;  // [n_seqs] the lowest child of each row
    int* staged_table;  // copies of table and lens where the outputs are in their place
    int* staged_lens;
    int* place;   // [n_pages] where each page goes, -1 for free ones
    int* movers;  // [n_pages / 2] pages that move, the last one first

    __device__ __forceinline__ int held(int len) const {
        return (int)(((long long)len + (1 << page_shift) - 1) >> page_shift);
    }
    __device__ __forceinline__ bool names(int v) const { return v >= 0 && v < n_pages; }
};

// One cluster's threads, and sums over its warps.
struct Team {
    cg::cluster_group cluster = cg::this_cluster();
    int rank, ctas, warp, lane, id;
    int* sums;  // [kWarps] of this CTA
    bool bad = false;

    __device__ explicit Team(int* shared_sums) : sums(shared_sums) {
        rank = (int)cluster.block_rank();
        ctas = (int)cluster.num_blocks();
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        id = rank * kWarps + warp;
    }
    __device__ void sync() {
        __threadfence();
        cluster.sync();
    }
    // This warp's part of [0, n), in pieces of 32.
    struct Slice {
        long long from, to;
    };
    __device__ Slice slice(long long n) const {
        const long long warps = (long long)ctas * kWarps;
        const long long each = ((n + 31) / 32 + warps - 1) / warps * 32;
        const long long from = min(n, each * id);
        return {from, min(n, from + each)};
    }
    // Sum of `x` (one number a warp) over the warps before this one; `total` over all.
    // Ends with everybody past its reads.
    __device__ int before(int x, int& total) {
        if (lane == 0) sums[warp] = x;
        sync();
        int mine = 0, all = 0;
        for (int r = 0; r < ctas; ++r) {
            const int* theirs = cluster.map_shared_rank(sums, r);
            const int y = theirs[lane];
            const int s = __reduce_add_sync(0xffffffffu, y);
            if (r < rank) mine += s;
            if (r == rank) mine += __reduce_add_sync(0xffffffffu, lane < warp ? y : 0);
            all += s;
        }
        total = all;
        sync();
        return mine;
    }
    __device__ void report(unsigned bits) {
        if (bits) atomicOr(&g_pages_status, bits);
    }
};

// Free pages in order: the i-th of them, i < wanted, goes to got[i] and is counted as
// named once.  Returns how many there are, at most `wanted`.
__device__ int take_free(Team& t, const PageArgs& a, int wanted) {
    const Team::Slice s = t.slice(a.n_pages);
    int mine = 0;
    for (long long i = s.from + t.lane; i < s.to; i += 32) mine += __ldcg(a.refs_out + i) <= 0;
    mine = __reduce_add_sync(0xffffffffu, mine);
    int total, at = t.before(mine, total);
    if (mine) {
        for (long long i0 = s.from; i0 < s.to && at < wanted; i0 += 32) {
            const long long i = i0 + t.lane;
            const bool free = i < s.to && __ldcg(a.refs_out + i) <= 0;
            const unsigned all = __ballot_sync(0xffffffffu, free);
            const int n = at + __popc(all & ((1u << t.lane) - 1));
            if (free && n < wanted) {
                a.got[n] = (int)i;
                a.refs_out[i] = 1;
            }
            at += __popc(all);
        }
    }
    t.sync();
    return min(total, wanted);
}

__device__ __forceinline__ int clamped_len(const PageArgs& a, int len, unsigned& bad) {
    const long long most = (long long)a.width << a.page_shift;
    if (len < 0 || len > most) bad |= STATUS_BAD_PAGES;
    return (int)min(max((long long)len, 0LL), most);
}

__global__ void __launch_bounds__(kThreads) resize_kernel(PageArgs a) {
    __shared__ int sums[32];
    Team t(sums);
    pdl_wait();
    pdl_release();
    unsigned bad = 0;
    const Team::Slice s = t.slice((long long)a.n_seqs * a.width);
    // entries past a sequence's length give their pages up; missing ones are counted
    int mine = 0;
    for (long long i = s.from + t.lane; i < s.to; i += 32) {
        const int n = (int)(i / a.width), col = (int)(i - (long long)n * a.width);
        const int v = a.table_out[i];
        if (v < -1 || v >= a.n_pages) bad |= STATUS_BAD_PAGES;
        if (col < a.held(clamped_len(a, __ldcg(a.lens + n), bad))) {
            mine += !a.names(v);
        } else if (v != -1) {
            if (a.names(v)) atomicAdd(a.refs_out + v, -1);
            a.table_out[i] = -1;
        }
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    int wanted, at = t.before(mine, wanted);
    if (wanted) {
        const int there = take_free(t, a, wanted);
        if (there < wanted) bad |= STATUS_NO_PAGES;
        if (mine) {
            for (long long i0 = s.from; i0 < s.to; i0 += 32) {
                const long long i = i0 + t.lane;
                bool miss = false;
                if (i < s.to) {
                    const int n = (int)(i / a.width), col = (int)(i - (long long)n * a.width);
                    unsigned ignore = 0;
                    miss = col < a.held(clamped_len(a, __ldcg(a.lens + n), ignore)) &&
                           !a.names(a.table_out[i]);
                }
                const unsigned all = __ballot_sync(0xffffffffu, miss);
                const int k = at + __popc(all & ((1u << t.lane) - 1));
                if (miss) a.table_out[i] = k < there ? __ldcg(a.got + k) : -1;
                at += __popc(all);
            }
        }
    }
    t.report(bad);
}

__global__ void __launch_bounds__(kThreads) fork_kernel(PageArgs a) {
    __shared__ int sums[32];
    Team t(sums);
    pdl_wait();
    pdl_release();
    unsigned bad = 0;
    const int threads = t.ctas * kThreads, me = t.rank * kThreads + threadIdx.x;
    const long long entries = (long long)a.n_seqs * a.width;
    const int *table = a.table, *lens = a.lens;
    if (a.table == a.table_out) {
        for (long long i = me; i < entries; i += threads) a.staged_table[i] = a.table[i];
        table = a.staged_table;
    }
    if (a.lens == a.lens_out) lens = a.staged_lens;
    if (a.refs != a.refs_out)
        for (int i = me; i < a.n_pages; i += threads) a.refs_out[i] = a.refs[i];
    for (int n = me; n < a.n_seqs; n += threads) {
        a.first[n] = a.n_seqs;
        if (a.lens == a.lens_out) a.staged_lens[n] = a.lens[n];
    }
    t.sync();
    auto parent_of = [&](int n) {
        const int p = __ldcg(a.parent + n);
        if (p < -1 || p >= a.n_seqs) bad |= STATUS_BAD_PAGES;
        return p >= 0 && p < a.n_seqs ? p : -1;
    };
    for (int n = me; n < a.n_seqs; n += threads) {
        const int p = parent_of(n);
        if (p >= 0) atomicMin(a.first + p, n);
    }
    t.sync();
    // whether row n has a last page of its own to get; its parent's length
    auto copied = [&](int n, int p, int& len) {
        len = p < 0 ? 0 : clamped_len(a, __ldcg(lens + p), bad);
        return p >= 0 && (len & ((1 << a.page_shift) - 1)) && __ldcg(a.first + p) != n;
    };
    for (long long i = me; i < entries; i += threads) {
        const int n = (int)(i / a.width), col = (int)(i - (long long)n * a.width);
        const int p = parent_of(n);
        int len;
        const bool copy = copied(n, p, len);
        const int held = a.held(len), old = __ldcg(table + i);
        if (old < -1 || old >= a.n_pages) bad |= STATUS_BAD_PAGES;
        int now = -1;
        if (col < held - (copy ? 1 : 0)) now = __ldcg(table + (long long)p * a.width + col);
        if (!a.names(now)) now = -1;
        if (old != now) {
            if (a.names(old)) atomicAdd(a.refs_out + old, -1);
            if (now >= 0) atomicAdd(a.refs_out + now, 1);
        }
        a.table_out[i] = now;
    }
    // pages for the copies, in the order of their rows
    const Team::Slice s = t.slice(a.n_seqs);
    int mine = 0;
    for (long long n = s.from + t.lane; n < s.to; n += 32) {
        int len;
        mine += copied((int)n, parent_of((int)n), len);
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    int wanted, at = t.before(mine, wanted);
    const int there = wanted ? take_free(t, a, wanted) : 0;
    if (there < wanted) bad |= STATUS_NO_PAGES;
    for (long long n0 = s.from; n0 < s.to; n0 += 32) {
        const long long n = n0 + t.lane;
        int len = 0, p = -1;
        bool copy = false;
        if (n < s.to) copy = copied((int)n, p = parent_of((int)n), len);
        const unsigned all = __ballot_sync(0xffffffffu, copy);
        const int k = at + __popc(all & ((1u << t.lane) - 1));
        at += __popc(all);
        if (copy) {
            const int last = a.held(len) - 1;
            if (k < there) {
                const int page = __ldcg(a.got + k);
                a.table_out[n * a.width + last] = page;
                a.src[k] = __ldcg(table + (long long)p * a.width + last);
                a.dst[k] = page;
            } else {
                len = last << a.page_shift;
            }
        }
        if (n < s.to) {
            a.lens_out[n] = len;
            if (n >= there) a.src[n] = a.dst[n] = -1;
        }
    }
    if (me == 0) a.count[0] = there;
    t.report(bad);
}

__global__ void __launch_bounds__(kThreads) compact_kernel(PageArgs a) {
    __shared__ int sums[32];
    Team t(sums);
    pdl_wait();
    pdl_release();
    unsigned bad = 0;
    const int threads = t.ctas * kThreads, me = t.rank * kThreads + threadIdx.x;
    const Team::Slice s = t.slice(a.n_pages);
    int mine = 0;
    for (long long i = s.from + t.lane; i < s.to; i += 32) mine += a.refs[i] > 0;
    mine = __reduce_add_sync(0xffffffffu, mine);
    int used, before = t.before(mine, used);
    // holes, below `used`; pages to move, from there on, counted from the end
    int at = before;
    for (long long i0 = s.from; i0 < s.to; i0 += 32) {
        const long long i = i0 + t.lane;
        const int count = i < s.to ? a.refs[i] : 0;
        const unsigned all = __ballot_sync(0xffffffffu, count > 0);
        const int below = at + __popc(all & ((1u << t.lane) - 1));  // pages in use before i
        at += __popc(all);
        if (i >= s.to) continue;
        a.place[i] = count > 0 ? (int)i : -1;
        if (i < used && count <= 0) a.dst[i - below] = (int)i;
        if (i >= used && count > 0) a.movers[used - 1 - below] = (int)i;
        if (a.refs != a.refs_out) a.refs_out[i] = count;
    }
    t.sync();
    // how many: pages in use from `used` on, one for each hole
    int high = 0;
    for (long long i = max(s.from, (long long)used) + t.lane; i < s.to; i += 32)
        high += __ldcg(a.refs + i) > 0;
    high = __reduce_add_sync(0xffffffffu, high);
    int moved;
    t.before(high, moved);
    for (int k = me; k < a.n_pages / 2; k += threads) {
        if (k < moved) {
            const int from = __ldcg(a.movers + moved - 1 - k), to = __ldcg(a.dst + k);
            a.src[k] = from;
            a.refs_out[to] = __ldcg(a.refs + from);
        } else {
            a.src[k] = a.dst[k] = -1;
        }
    }
    t.sync();
    for (int k = me; k < moved; k += threads) {
        const int from = __ldcg(a.src + k);
        a.refs_out[from] = 0;
        a.place[from] = __ldcg(a.dst + k);
    }
    t.sync();
    const long long entries = (long long)a.n_seqs * a.width;
    for (long long i = me; i < entries; i += threads) {
        const int v = a.table[i];
        if (v < -1 || v >= a.n_pages) bad |= STATUS_BAD_PAGES;
        // (an entry whose page is free by its count names none)
        const int now = a.names(v) ? __ldcg(a.place + v) : -1;
        if (a.names(v) && now < 0) bad |= STATUS_BAD_PAGES;
        a.table_out[i] = now;
    }
    if (me == 0) a.count[0] = moved;
    t.report(bad);
}

// Pages move in pieces of 16 KB, a CTA each, four 16-byte loads a thread in flight.
constexpr int kCopyThreads = 256;
constexpr int kPiece = 16384;
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
    const long long total = (long long)pairs * n_caches * pieces;
    for (long long i = blockIdx.x; i < total; i += gridDim.x) {
        const long long page = i / pieces, pair = page / n_caches;
        const int s = __ldcg(src + pair), d = __ldcg(dst + pair);
        if (s < 0 || s >= n_pages || d < 0 || d >= n_pages) {
            if (threadIdx.x == 0) atomicOr(&g_pages_status, STATUS_BAD_PAGES);
            continue;
        }
        uint8_t* cache = caches.at[page - pair * n_caches];
        const long long from = (i - page * pieces) * kPiece;
        const int n = (int)(min((long long)kPiece, page_bytes - from) / 16);
        const uint4* x = reinterpret_cast<const uint4*>(cache + s * page_bytes + from);
        uint4* y = reinterpret_cast<uint4*>(cache + d * page_bytes + from);
        constexpr int kEach = kPiece / 16 / kCopyThreads;
        uint4 u[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (threadIdx.x + e * kCopyThreads < n) u[e] = __ldcs(x + threadIdx.x + e * kCopyThreads);
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (threadIdx.x + e * kCopyThreads < n) __stcs(y + threadIdx.x + e * kCopyThreads, u[e]);
    }
}

struct Layout {
    size_t got, first, table, lens, place, movers, bytes;
};
Layout workspace_layout(long long n_pages, long long n_seqs, long long width) {
    auto round = [](long long ints) { return (size_t)((ints * 4 + 15) / 16 * 16); };
    Layout l;
    l.got = 0;
    l.first = l.got + round(n_pages);
    l.table = l.first + round(n_seqs);
    l.lens = l.table + round(n_seqs * width);
    l.place = l.lens + round(n_seqs);
    l.movers = l.place + round(n_pages);
    l.bytes = l.movers + round(n_pages / 2);
    return l;
}

bool int_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

kda_status pages_call(const char* fn, void (*kernel)(PageArgs), PageArgs a, int64_t n_pages,
                      int page, void* workspace, size_t workspace_bytes, uint64_t stream) {
    KDA_REQUIRE(page == 16 || page == 32 || page == 64 || page == 128 || page == 256,
                KDA_ERR_UNSUPPORTED, "%s: pages of %d tokens (only 16, 32, 64, 128, 256)", fn,
                page);
    KDA_REQUIRE(a.n_seqs >= 1 && a.width >= 1 && a.width <= 0x7fffffff / page && n_pages >= 1 &&
                    n_pages < 0x7fffffff,
                KDA_ERR_INVALID_ARG,
                "%s: n_seqs (%d), max_pages (%d) and n_pages (%lld) must be positive, max_pages "
                "* page and n_pages below 2^31",
                fn, a.n_seqs, a.width, (long long)n_pages);
    KDA_REQUIRE((long long)a.n_seqs * a.width < 0x7fffffffLL, KDA_ERR_INVALID_ARG,
                "%s: a page table of 2^31 entries or more", fn);
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
    a.got = reinterpret_cast<int*>(ws + l.got);
    a.first = reinterpret_cast<int*>(ws + l.first);
    a.staged_table = reinterpret_cast<int*>(ws + l.table);
    a.staged_lens = reinterpret_cast<int*>(ws + l.lens);
    a.place = reinterpret_cast<int*>(ws + l.place);
    a.movers = reinterpret_cast<int*>(ws + l.movers);
    // a CTA for every 4096 integers, within a cluster's limit
    const long long ints = n_pages + (long long)a.n_seqs * a.width;
    const int ctas = ints <= 4096 ? 1 : ints <= 8192 ? 2 : ints <= 16384 ? 4 : kMostCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = as_stream(stream);
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
    if (n_pages < 1 || n_pages >= 0x7fffffff || n_seqs < 1 || max_pages < 1 ||
        (long long)n_seqs * max_pages >= 0x7fffffffLL)
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
    const unsigned grid = (unsigned)(most < 152 * 8 ? most : 152 * 8);
    launch_pdl(copy_kernel, dim3(grid), dim3(kCopyThreads), 0, as_stream(stream), c, n_caches,
               (long long)n_pages, bytes, src, dst, count, max_count);
    return launch_result(fn);
}
