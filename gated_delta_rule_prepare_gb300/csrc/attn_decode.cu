// Attention of 1..8 query rows per sequence over the paged 4-bit cache
// (kda_attn_kv4_decode): kda_attn_prefill's formula with the cache's values
// m + s * code as keys and values.
//
// HBM-bound: 144 bytes per (position, KV head), read once for all of the
// group's query heads and rows.  What the values cost on the way:
//  - Codes go to the matrix instructions as they are: with 64 channels to a
//    step s and a minimum m,
//        q . k = sum_a s_a (q . code)_a + m_a (sum q)_a
//        o_d   = sum_t (p_t s_ta) (code - 8)_td + sum_t p_t (m_ta + 8 s_ta)
//    so steps and minima meet scores and weights, not values.  Four bits at the
//    low end of an FP16 number are a subnormal, code * 2^-24, the next four
//    code * 2^-20: one AND makes two operands, and the powers of two go into q
//    and the output.
//  - The cache keeps codes in the order of mma.sync's A operand, which is also
//    that of two B operands: up to 8 queries are the 8 columns of the products
//    (keys, or value channels, the 16 rows: attend_narrow), more are the 16 rows
//    (attend_wide).  Codes go from the copied page to registers, nothing is
//    transposed in shared memory.
//  - A score's place is its query's in the output too: running sums and rescaling
//    stay within a lane.  p_t s_ta is rounded to FP16 after a common power of two
//    that keeps it below 2^15 (11 significant bits; weights down to 2^-33 of the
//    largest); scores, sums and outputs are FP32.
// What bounds it then: four warps a scheduler (registers and the rings allow no
// more), in each of which the pages' arrival, unpacking and fixed latencies follow
// each other, so that issue is busy 54 to 57 % of the time and no stall stands out;
// in short segments, their starts and ends.  64 sequences of 2000 to 8192 tokens, 32
// heads over 8: 83.7 us, 4.4 TB/s; 128 sequences of 4 rows (16 queries a KV head):
// 143 us, 2.9 TB/s; one of 131000 tokens and 2 rows: 41 us.
//
// All positions of the batch, in chunks of 128 tokens, are one line that the
// CTAs cut into equal pieces, whatever the lengths: a piece ends where it ends,
// and what is left of a (sequence, head) in each is joined by a second kernel
// (attn_join_kernel), always in the same order.  Per CTA one warp copies chunks
// into a ring in shared memory and four attend over them.
#include <algorithm>
#include <cmath>

#include "attn_common.h"
#include "f32x2.h"
#include "sm103_tc.h"
#include "tma_map.h"

namespace kda {
namespace {

using namespace attn;
using tc::bulk_load;
using tc::fence_mbar_init;
using tc::mbar_arrive;
using tc::mbar_arrive_expect_tx;
using tc::mbar_init;
using tc::mbar_wait;

__device__ unsigned g_decode_status = 0;

// A chunk is 8 groups of 16 tokens; each of a CTA's four warps takes two.
// Several small CTAs to a multiprocessor, not one large one: while one ends a
// segment the others go on (one of 12 warps: 116 us at 64 sequences of 2000 to
// 8192 tokens, three of 4: 94.5).  A thread's registers hold all it has; what
// spills costs more than anything else here, as the rings leave next to no L1
// cache.
constexpr int kWarps = 4;  // and one that copies
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kCtas = 3;  // to a multiprocessor
constexpr int kStages = 3;
constexpr int kGroups = 8;
constexpr int kChunk = kGroups * 16;  // tokens
constexpr int kStageBytes = kChunk * kTokenBytes;
// Query rows of a block: where a KV head has up to 8 they are the columns of
// the products with 16 keys, else 16 of them are the rows of the products with
// 8 keys.
template <bool WIDE>
constexpr int kRows = WIDE ? 16 : 8;
// What a segment's start and end cost, in chunks: pieces are cut with it (128
// sequences of 4 rows and 100 to 6000 tokens, many of a chunk or two: with 0, 182
// us; 1, 161; 2, 148; 3, 142; 4, 144; 6, 150.  64 sequences of 2000 to 8192: 91.8,
// 89.5, 88.1, 88.1, 89.7, 90.9).
constexpr int kExtra = 3;

struct DecodeArgs {
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    int n_seqs, krows, heads, window;
    int reach;  // how many last positions some row may see: 2^31 - 1 without a window
    int group, rows, blocks;  // heads per KV head; query rows of a KV head; blocks of them
    float scale;
    int pieces;  // CTAs of the main kernel
    float* part;  // [2 * pieces][query row][128] sums, then [2 * pieces][query row] (shift, l)
    struct Job* jobs;
    Cache c;
};
// What there is to join: the pieces first..last share a (sequence, head, block of
// query rows).  Of a piece b, part 2 b is of the one that it starts within, part
// 2 b + 1 of one that starts in it and goes on.  A job for each (sequence, head,
// block) where there are no more than pieces, else for what goes on from a piece.
struct Job {
    int n, unit, first, last;
};
__device__ __forceinline__ bool job_a_unit(const DecodeArgs& a) {
    return (long long)a.n_seqs * a.c.kv_heads * a.blocks <= a.pieces;
}

// Chunks that sequence n's queries see: [first, first + count).
struct Chunks {
    int first, count;
};
__device__ __forceinline__ int good_len(const DecodeArgs& a, int len) {
    return len < 0 || (long long)len > ((long long)a.c.max_pages << a.c.page_shift) ? 0 : len;
}
__device__ __forceinline__ Chunks chunks_of(const DecodeArgs& a, int len) {
    const int lo = max(0, len - a.reach) / kChunk;
    return {lo, len > 0 ? (len - 1) / kChunk + 1 - lo : 0};
}
// (64-bit divisions are long: most need 32 bits.)
__device__ __forceinline__ long long divide(long long x, long long y) {
    if (((x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
    return x / y;
}
// What a (head, block) of a sequence is on the line: its chunks, behind kExtra
// places that stand for the cost of a segment's start and end.
__device__ __forceinline__ int places(const DecodeArgs& a, const Chunks& ch) {
    return ch.count ? ch.count + kExtra : 0;
}
// The line of `total` places is cut into pieces of `size`, the last one shorter;
// piece b is CTA b's.
__device__ __forceinline__ long long piece_size(const DecodeArgs& a, long long total) {
    return divide(total + a.pieces - 1, a.pieces);
}

// All lengths by one warp: the places of all sequences of one (head, block),
// and, through `each`, those before sequences n..n + 31 (lane by lane).
template <class Each>
__device__ __forceinline__ long long scan_lengths(const DecodeArgs& a, Each each) {
    const int lane = threadIdx.x & 31;
    long long before = 0;
    for (int n0 = 0; n0 < a.n_seqs; n0 += 256) {
        int len[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = n0 + 32 * i + lane;
            len[i] = n < a.n_seqs ? __ldg(a.c.lens + n) : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (n0 + 32 * i >= a.n_seqs) break;
            const int mine = places(a, chunks_of(a, good_len(a, len[i])));
            int sum = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += up;
            }
            if (!each(n0 + 32 * i, before + sum - mine, mine)) return before;
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    return before;
}

// What a stage of the ring holds.  A segment is what one CTA does of one
// (sequence, head, block of query rows).
struct Stage {
    int pos;         // the chunk's first position
    uint32_t flags;  // bit i: tokens 16 i .. 16 i + 15 are in the stage; then:
    int len;         // of the sequence
    int n, head, block;
    int part;  // where an incomplete segment's sums go, or -1
};
constexpr uint32_t kStart = 1u << 24, kEnd = 1u << 25, kNoMore = 1u << 26;

constexpr int kPad = 132;  // a query's 128 sums, so that a warp's stores meet all banks
constexpr int kBuffers = 2;  // two warps' each
static_assert(kWarps == 2 * kBuffers, "");
template <bool WIDE>
struct Shared {
    uint64_t full[kStages], empty[kStages];
    Stage stage[kStages];
    // by query, the factor from a product to a score in log2 units, the sums over
    // 64 channels, and the first position that is not seen
    float unit[kRows<WIDE>];
    float2 qsum[kRows<WIDE>];
    int limit[kRows<WIDE>];
    // a segment's end
    float2 stat[kWarps][kRows<WIDE>];  // a warp's (shift, l) by query
    union {
        // the segment's queries as operands (FP16, scaled by a power of two)
        alignas(16) uint32_t q[8][32][WIDE ? 4 : 2];
        // and at its end the warps' outputs
        alignas(16) float sums[kBuffers][kRows<WIDE>][kPad];
    };
    int stop;
};
template <bool WIDE>
constexpr int smem_bytes() {
    return kStages * kStageBytes + (int)sizeof(Shared<WIDE>);
}

template <bool B>
struct Bool {
    static constexpr bool value = B;
};

// Waits end: with the phase, with another role's giving up, or after 2^33 clocks.
__device__ __forceinline__ bool wait_more(uint64_t* bar, uint32_t parity, int* stop) {
    const long long from = clock64();
    while (!mbar_wait(bar, parity, 32)) {
        if (*(volatile int*)stop) return false;
        if (clock64() - from > 1LL << 33) {
            atomicOr(&g_decode_status, STATUS_TIMEOUT);
            *(volatile int*)stop = 1;
            return false;
        }
    }
    return true;
}
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, int* stop) {
    return wait_more(bar, parity, stop);
}
// The long wait is a function of its own, out of the instruction cache's way (64
// sequences of 2000 to 8192 tokens: 88.1 us with it in the loops, 84.3), but not
// where that makes registers spill (128 of 4 rows: 142 us, as a function 150).
template <bool WIDE>
__device__ __forceinline__ bool wait_warp(Shared<WIDE>& sh, uint64_t* bar, uint32_t parity) {
    bool ok = mbar_wait(bar, parity, 1);
    if (!ok) ok = WIDE ? wait_more(bar, parity, &sh.stop) : wait_long(bar, parity, &sh.stop);
    return __all_sync(0xffffffffu, ok);
}

// Tokens that lie together in the cache and in a stage: a stage holds pieces of
// so many, each laid out as a page of its size, so that a page of up to 128
// tokens is one copy.  (Small copies cost what large ones do: with four to a
// page, codes and parameters apart, copying alone took 75 us where it takes 66 to
// 68, 64 sequences of 2000 to 8192 tokens.)
__device__ __forceinline__ int piece_tokens(const DecodeArgs& a) { return min(a.c.page(), 128); }

// Where a stage's group of 16 tokens has its codes and parameters of K; those of
// V are part_bytes(piece_tokens) further.
__device__ __forceinline__ void group_places(const DecodeArgs& a, int group, int& codes_at,
                                             int& pars_at) {
    const int tok = group * 16, piece = piece_tokens(a);
    const int in = tok & (piece - 1), block = (tok - in) * kTokenBytes;
    codes_at = block + in * 64;
    pars_at = block + piece * 64 + in * 8;
}

__device__ __forceinline__ void prefetch_l1(const void* p) {
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}
// What the consumers will want of the segment's queries, 128 bytes a lane.
template <bool WIDE>
__device__ __forceinline__ void touch_queries(const DecodeArgs& a, int n, int head, int block) {
    const int lane = threadIdx.x & 31;
    const int row = block * kRows<WIDE> + (lane >> 1), i = row / a.group;
    if ((lane >> 1) < kRows<WIDE> && row < a.rows)
        prefetch_l1(a.q + (((long long)n * a.krows + i) * a.heads + head * a.group + row -
                           i * a.group) * D + 64 * (lane & 1));
}

// The copying warp: walks this CTA's piece of the line.
template <bool WIDE>
__device__ __forceinline__ void copy_role(const DecodeArgs& a, Shared<WIDE>& sh, uint8_t* sm) {
    const int lane = threadIdx.x & 31;
    const int heads = a.c.kv_heads, per_seq = heads * a.blocks;
    bool bad_len = false;
    const long long one = scan_lengths(a, [](int, long long, int) { return true; });
    const long long total = one * per_seq;
    const long long size = piece_size(a, total);
    const long long from = min(total, size * blockIdx.x), to = min(total, from + size);
    // the sequence that holds `from`, and where it starts
    int n = 0;
    long long n_start = 0;
    if (from < to)
        scan_lengths(a, [&](int n0, long long before, int mine) {
            const unsigned hit = __ballot_sync(
                0xffffffffu, before * per_seq <= from && (before + mine) * per_seq > from);
            if (!hit) return true;
            const int who = __ffs(hit) - 1;
            n = n0 + who;
            n_start = __shfl_sync(0xffffffffu, before, who) * per_seq;
            return false;
        });
    if (blockIdx.x == 0) {
        for (int i = lane; i < a.n_seqs; i += 32) {
            const int len = __ldg(a.c.lens + i);
            bad_len |= len != good_len(a, len);
        }
        if (bad_len) atomicOr(&g_decode_status, STATUS_BAD_PAGES);
    }
    const bool by_unit = job_a_unit(a);
    if (lane == 0 && !by_unit) a.jobs[blockIdx.x] = {0, 0, 0, -1};
    // sequences that nothing is seen of
    for (int i = blockIdx.x; i < a.n_seqs; i += a.pieces) {
        if (chunks_of(a, good_len(a, __ldg(a.c.lens + i))).count) continue;
        const long long row = (long long)i * a.krows * a.heads;
        for (int k = 0; k < a.krows * a.heads; ++k)
            reinterpret_cast<uint2*>(a.o + (row + k) * D)[lane] = make_uint2(0u, 0u);
        if (a.lse)
            for (int k = lane; k < a.krows * a.heads; k += 32) a.lse[row + k] = -INFINITY;
        if (by_unit)
            for (int k = lane; k < per_seq; k += 32)
                a.jobs[i * per_seq + k] = {i, k, 0, -1};
    }
    int stage = 0;
    uint32_t phase = 0;
    bool go = true;
    // a chunk's pieces, and bits of `flags` for one
    const int piece = piece_tokens(a);
    const int per_chunk = kChunk / piece;
    const uint32_t groups = (1u << (piece / 16)) - 1;
    long long at = from;
    while (go && at < to) {
        const int len = good_len(a, __ldg(a.c.lens + n));
        const Chunks ch = chunks_of(a, len);
        const int length = places(a, ch);
        // (n, head, block) units of this sequence, chunk by chunk
        while (go && at < to && at < n_start + (long long)length * per_seq) {
            const int unit = (int)divide(at - n_start, length);
            const int head = unit / a.blocks, block = unit - head * a.blocks;
            const long long u_start = n_start + (long long)unit * length + kExtra;
            const long long u_end = u_start + ch.count;
            const long long seg_end = min(u_end, to);
            at = max(at, u_start);
            if (at >= to) break;
            const bool starts = at == u_start, whole = starts && seg_end == u_end;
            const int part = whole ? -1 : 2 * (int)blockIdx.x + (starts ? 1 : 0);
            const long long seg_start = at;
            if (lane == 0 && starts && (by_unit || !whole)) {
                const int first = (int)blockIdx.x;
                const int last = whole ? -1 : (int)divide(u_end - 1, size);
                a.jobs[by_unit ? n * per_seq + unit : first] = {n, unit, first, last};
            }
            const int* table = a.c.table + (long long)n * a.c.max_pages;
            touch_queries<WIDE>(a, n, head, block);
            if (n + 1 < a.n_seqs && lane == 0) prefetch_l1(table + a.c.max_pages);
            // page numbers, a lane each, some chunks ahead
            int ids = 0, ids_from = -1;
            for (; go && at < seg_end; ++at) {
                const int chunk = ch.first + (int)(at - u_start);
                const int pos = chunk * kChunk;
                const int at_tok = pos + lane * piece;  // this lane's piece
                const bool wanted = lane < per_chunk && at_tok < len;
                const int last_page = (pos + kChunk - 1) >> a.c.page_shift;
                if (ids_from < 0 || last_page >= ids_from + 32) {
                    ids_from = pos >> a.c.page_shift;
                    const int p = ids_from + lane;
                    ids = p < a.c.max_pages && ((long long)p << a.c.page_shift) < len
                              ? __ldg(table + p)
                              : -1;
                }
                const int id =
                    __shfl_sync(0xffffffffu, ids, (at_tok >> a.c.page_shift) - ids_from);
                const bool valid = wanted && id >= 0 && id < a.c.n_pages;
                if (wanted && !valid) atomicOr(&g_decode_status, STATUS_BAD_PAGES);
                const unsigned ok = __ballot_sync(0xffffffffu, valid);
                uint32_t there = 0;
                for (int i = 0; i < per_chunk; ++i)
                    if (ok >> i & 1) there |= groups << (i * (piece / 16));
                go = wait_warp(sh, &sh.empty[stage], phase ^ 1);
                if (!go) break;
                if (lane == 0) {
                    if (at == seg_start) there |= kStart;
                    if (at + 1 == seg_end) there |= kEnd;
                    sh.stage[stage] = {pos, there, len, n, head, block, part};
                    mbar_arrive_expect_tx(&sh.full[stage],
                                          (uint32_t)__popc(ok) * piece * kTokenBytes);
                }
                __syncwarp();
                if (valid) {
                    const int in_page = at_tok & (a.c.page() - 1);
                    const uint8_t* src = a.c.data +
                                         ((long long)id * heads + head) * a.c.block_bytes();
                    uint8_t* dst = sm + stage * kStageBytes + lane * piece * kTokenBytes;
                    if (piece == a.c.page()) {
                        bulk_load(dst, src, piece * kTokenBytes, &sh.full[stage]);
                    } else {
                        const int page = a.c.page();
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            const uint8_t* half = src + v * part_bytes(page);
                            bulk_load(dst + v * part_bytes(piece), half + in_page * 64, piece * 64,
                                      &sh.full[stage]);
                            bulk_load(dst + v * part_bytes(piece) + piece * 64,
                                      half + page * 64 + in_page * 8, piece * 8, &sh.full[stage]);
                        }
                    }
                }
                __syncwarp();
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
        }
        n_start += (long long)length * per_seq;
        ++n;
    }
    if (go) go = wait_warp(sh, &sh.empty[stage], phase ^ 1);
    if (lane == 0) {
        if (go) {
            sh.stage[stage].flags = kNoMore;
            mbar_arrive(&sh.full[stage]);
        } else {
            // copies in flight land before the CTA's memory goes away
            for (int s = 0; s < kStages; ++s)
                mbar_wait(&sh.full[s], s < stage ? phase : phase ^ 1, 1 << 12);
        }
    }
}

// A word of codes as the A operand: FP16 numbers code * 2^-24 (from the low
// four bits of a byte) and code * 2^-20.
__device__ __forceinline__ void codes(uint32_t w, uint32_t& lo0, uint32_t& hi0, uint32_t& lo1,
                                      uint32_t& hi1) {
    lo0 = w & 0x000f000fu;
    hi0 = w & 0x00f000f0u;
    lo1 = w >> 8 & 0x000f000fu;
    hi1 = w >> 8 & 0x00f000f0u;
}
__device__ __forceinline__ uint32_t sub_h2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
constexpr float kLow = 16777216.f, kHigh = 1048576.f;  // 2^24, 2^20
// The same of code - 8: a rounding of a weight then meets at most eight steps.
__device__ __forceinline__ void centred_codes(uint32_t w, uint32_t& lo0, uint32_t& hi0,
                                              uint32_t& lo1, uint32_t& hi1) {
    codes(w, lo0, hi0, lo1, hi1);
    lo0 = sub_h2(lo0, 0x00080008u);  // 8 * 2^-24
    hi0 = sub_h2(hi0, 0x00800080u);  // 8 * 2^-20
    lo1 = sub_h2(lo1, 0x00080008u);
    hi1 = sub_h2(hi1, 0x00800080u);
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit elements, a row to four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void consumer_sync() {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
}
// Over the eight lanes that hold the other keys of the same queries.
__device__ __forceinline__ float sum_keys(float x) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}
__device__ __forceinline__ float max_keys(float x) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    return x;
}

__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
    return __uint_as_float((uint32_t)(127 + e) << 23);
}
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23 & 255) - 127; }

// The segment's queries to operands: some rows a warp, four channels a lane.
template <bool F16, bool WIDE>
__device__ __forceinline__ void load_queries(const DecodeArgs& a, Shared<WIDE>& sh,
                                             const Stage& st) {
    constexpr int N = kRows<WIDE> / kWarps;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint2 rows[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int row = st.block * kRows<WIDE> + warp + kWarps * k, i = row / a.group;
        rows[k] = make_uint2(0u, 0u);
        if (row < a.rows)
            rows[k] = __ldg(reinterpret_cast<const uint2*>(
                                a.q + (((long long)st.n * a.krows + i) * a.heads +
                                       st.head * a.group + row - i * a.group) * D) + lane);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int r = warp + kWarps * k;
        const uint2 raw = rows[k];
        float2 x = widen2<F16>(raw.x), y = widen2<F16>(raw.y);
        float big = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y)));
#pragma unroll
        for (int off = 1; off < 32; off <<= 1)
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
        // bring the largest to 2^14..2^15: exact, and what is below FP16's
        // smallest number then is 2^-34 of it
        const bool plain = big == 0.f || !(big < INFINITY);
        const int up = plain ? 0 : max(-126, min(126, 14 - exponent(big)));
        const float f = pow2(up);
        x.x *= f, x.y *= f, y.x *= f, y.y *= f;
        float sum = (x.x + x.y) + (y.x + y.y);
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        // channel 16 kb + 8 j + 2 t + e: codes of j = 1 are the high four bits
        const int kb = lane >> 2, j = lane >> 1 & 1, t0 = 2 * (lane & 1);
        const float fj = j ? kHigh / kLow : 1.f;
        const int word = WIDE ? (r >> 3) + 2 * j : j, at = (r & 7) * 4 + t0;
        sh.q[kb][at][word] = narrow2<true>(x.x * fj, x.y * fj);
        sh.q[kb][at + 1][word] = narrow2<true>(y.x * fj, y.y * fj);
        if (lane == 0) {
            const int row = st.block * kRows<WIDE> + r;
            sh.limit[r] = row < a.rows ? max(0, st.len - a.krows + row / a.group + 1) : 0;
            sh.unit[r] = a.scale * kLog2e * kLow * pow2(-up);
            sh.qsum[r].x = sum * (1.f / kLow);
        }
        if (lane == 16) sh.qsum[r].y = sum * (1.f / kLow);
    }
    consumer_sync();
}

// The segment's end: the warps' sums, whose (shift, l) are in sh.stat, become one
// and go out.  `put` writes a warp's outputs, brought to the common shift, into a
// buffer, or adds them to what is there.
template <bool WIDE>
__device__ __forceinline__ float2 joint_stat(const Shared<WIDE>& sh, int c) {
    // the least shift is that of the largest score
    float least = INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (sh.stat[w][c].y != 0.f) least = fminf(least, sh.stat[w][c].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float2 x = sh.stat[w][c];
        if (x.y != 0.f) sum = fmaf(x.y, ex2_approx(least - x.x), sum);
    }
    return make_float2(least, sum);
}
template <bool F16, bool WIDE, class Put>
__device__ __forceinline__ void finish_segment(const DecodeArgs& a, Shared<WIDE>& sh,
                                               const Stage& st, Put put) {
    constexpr int Q = kRows<WIDE>, B = kBuffers;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    consumer_sync();
    if (warp < B) put(sh.sums[warp], Bool<false>{});
    consumer_sync();
    if (warp >= B) put(sh.sums[warp - B], Bool<true>{});
    consumer_sync();
    constexpr int kQuads = Q * 32 / (kWarps * 32);
    float4 all[kQuads];  // four channels of a query
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
        const float4 x = reinterpret_cast<const float4*>(sh.sums[0][warp + kWarps * i])[lane];
        const float4 y = reinterpret_cast<const float4*>(sh.sums[1][warp + kWarps * i])[lane];
        all[i] = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
    // (now: kept from before, they would spill)
    float2 stat[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) stat[i] = joint_stat(sh, warp + kWarps * i);
    consumer_sync();
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
        const int c = warp + kWarps * i, row = st.block * Q + c;
        const float2 joint = stat[i];
        const float4 x = all[i];
        if (st.part >= 0) {
            const long long at = (long long)st.part * Q + c;
            reinterpret_cast<float4*>(a.part)[at * 32 + lane] = x;
            if (lane == 0) reinterpret_cast<float2*>(a.part + 2LL * a.pieces * Q * D)[at] = joint;
        } else if (row < a.rows) {
            const float inv = joint.y == 0.f ? 0.f : 1.f / joint.y;
            const int i_row = row / a.group;
            const long long at = ((long long)st.n * a.krows + i_row) * a.heads +
                                 st.head * a.group + row - i_row * a.group;
            reinterpret_cast<uint2*>(a.o + at * D)[lane] =
                make_uint2(narrow2<F16>(x.x * inv, x.y * inv), narrow2<F16>(x.z * inv, x.w * inv));
            if (a.lse && lane == 0)
                a.lse[at] = joint.y == 0.f ? -INFINITY : (log2f(joint.y) - joint.x) * kLn2;
        }
    }
}

// A token's step and minimum of 64 channels.
__device__ __forceinline__ float step_of(uint32_t par) { return __uint_as_float(par << 16); }
__device__ __forceinline__ float least_of(uint32_t par) {
    return __uint_as_float(par & 0xffff0000u);
}

// What both forms keep of a query: weights are 2^(score + shift), at most 2^7; l
// sums them, moff weights times m + 8 s, by 64 channels.
struct Query {
    float shift, l, moff[2];
};
// What brings a warp's sums of query c to the common shift.
template <bool WIDE>
__device__ __forceinline__ float warp_factor(const Shared<WIDE>& sh, int c, const Query& q) {
    float least = INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (sh.stat[w][c].y != 0.f) least = fminf(least, sh.stat[w][c].x);
    return q.l != 0.f ? ex2_approx(least - q.shift) : 0.f;
}
// The power of two that steps enter with, below 2^8 then.  A segment begins with one
// so large that the first steps that are not zero bring it down, whichever rows of
// V have none.
struct Unit {
    float v = 0x1p120f;
    // for steps up to `most`; returns what that multiplies them by
    __device__ __forceinline__ float fit(float most) {
        const int was = exponent(v), now = max(-126, 6 - exponent(most));
        if (!(most > 0.f && most < INFINITY) || now + 2 > was) return 1.f;
        v = pow2(now);
        return pow2(max(-126, now - was));
    }
};

// Up to 8 queries, the columns 2 t + c of a lane; keys, and then value channels,
// are the 16 rows g and g + 8.  Two groups of 16 tokens at a time, so that their
// products and weights run in each other's waits.
template <bool F16>
__device__ __forceinline__ void attend_narrow(const DecodeArgs& a, Shared<false>& sh,
                                              const uint8_t* sm) {
    constexpr int I = 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int mine = I * warp;
    // where this warp's groups of a stage are: codes, parameters, of K; of V by
    // `to_v` further
    int codes_at[I], pars_at[I];
    const int to_v = part_bytes(piece_tokens(a));
#pragma unroll
    for (int u = 0; u < I; ++u) group_places(a, mine + u, codes_at[u], pars_at[u]);
    int stage = 0, len = 0;
    uint32_t phase = 0;
    uint2 qb[8];
    float unit[2], qsum[2][2], out[8][4];
    Query state[2];
    Unit v_unit;
    bool settled;  // every column has a shift that comes from a score
    int limit[2];  // positions from it on are not seen
    // (after a segment's end, not at the next one's start: it leaves the end their
    // registers)
    auto reset = [&] {
        settled = false;
        v_unit = {};
        state[0] = state[1] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k) qb[k] = make_uint2(0u, 0u);
#pragma unroll
        for (int c = 0; c < 2; ++c) unit[c] = qsum[c][0] = qsum[c][1] = 0.f, limit[c] = 0;
#pragma unroll
        for (int cb = 0; cb < 8; ++cb)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[cb][i] = 0.f;
    };
    reset();
    for (;;) {
        if (!wait_warp(sh, &sh.full[stage], phase)) return;
        const uint32_t flags = sh.stage[stage].flags;
        if (flags & kNoMore) return;
        if (flags & kStart) {
            const Stage st = sh.stage[stage];
            len = st.len;
            load_queries<F16>(a, sh, st);
#pragma unroll
            for (int k = 0; k < 8; ++k) qb[k] = *reinterpret_cast<const uint2*>(sh.q[k][lane]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                unit[c] = sh.unit[2 * t + c];
                qsum[c][0] = sh.qsum[2 * t + c].x;
                qsum[c][1] = sh.qsum[2 * t + c].y;
                limit[c] = sh.limit[2 * t + c];
            }
        }
        const uint32_t there = flags >> mine & ((1u << I) - 1);
        if (there) {
            const int pos = sh.stage[stage].pos + 16 * mine;
            const uint8_t* base = sm + stage * kStageBytes;
            // scores of tokens g and g + 8 of each group
            float y[I][4];
            {
                float acc[I][2][4] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int u = 0; u < I; ++u) {
                        const uint4 x =
                            reinterpret_cast<const uint4*>(base + codes_at[u])[lane + 32 * h];
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t ca[4];
                            codes(w[k], ca[0], ca[2], ca[1], ca[3]);
                            mma_f16(acc[u][h], ca, qb[4 * h + k].x, qb[4 * h + k].y);
                        }
                    }
#pragma unroll
                for (int u = 0; u < I; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint2 par =
                            reinterpret_cast<const uint2*>(base + pars_at[u])[g + 8 * i];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float d = least_of(par.x) * qsum[c][0];
                            d = fmaf(least_of(par.y), qsum[c][1], d);
                            d = fmaf(step_of(par.x), acc[u][0][2 * i + c], d);
                            d = fmaf(step_of(par.y), acc[u][1][2 * i + c], d);
                            y[u][2 * i + c] = fmaf(d, unit[c], state[c].shift);
                        }
                    }
            }
            // (a group that is not there, behind one that is, is masked whole)
            const bool edge = pos > len - a.krows + 1 - 16 * I ||
                              (a.window && pos < len - a.window) || there != (1u << I) - 1;
            if (edge) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int hi = limit[c], lo = a.window ? max(0, hi - a.window) : 0;
#pragma unroll
                    for (int u = 0; u < I; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int at = pos + 16 * u + g + 8 * i;
                            if (at < lo || at >= hi || !(there >> u & 1))
                                y[u][2 * i + c] = -INFINITY;
                        }
                }
            }
            uint2 vpar[I][2];
            float vs[I][2][2], most = 0.f;
#pragma unroll
            for (int u = 0; u < I; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    vpar[u][i] =
                        reinterpret_cast<const uint2*>(base + to_v + pars_at[u])[g + 8 * i];
                    vs[u][i][0] = step_of(vpar[u][i].x) * v_unit.v;
                    vs[u][i][1] = step_of(vpar[u][i].y) * v_unit.v;
                    // whatever the cache holds behind a sequence's end
                    if (edge && (pos + 16 * u + g + 8 * i >= len || !(there >> u & 1)))
                        vs[u][i][0] = vs[u][i][1] = 0.f;
                    most = fmaxf(most, fmaxf(vs[u][i][0], vs[u][i][1]));
                }
            float tops[2];
#pragma unroll
            for (int c = 0; c < 2; ++c)
                tops[c] = fmaxf(fmaxf(y[0][c], y[0][2 + c]), fmaxf(y[1][c], y[1][2 + c]));
            if (__any_sync(0xffffffffu,
                           !settled || most >= 256.f || tops[0] > 7.f || tops[1] > 7.f)) {
                // shifts: from the first scores of a column, and again once a
                // weight would pass 2^7; the steps' unit likewise (with the first one the
                // steps may have passed FP32's range: they are formed again)
                most = 0.f;
#pragma unroll
                for (int u = 0; u < I; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (vs[u][i][0] != 0.f) most = fmaxf(most, step_of(vpar[u][i].x));
                        if (vs[u][i][1] != 0.f) most = fmaxf(most, step_of(vpar[u][i].y));
                    }
                const float fv = v_unit.fit(max_keys(most));
#pragma unroll
                for (int u = 0; u < I; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (vs[u][i][0] != 0.f) vs[u][i][0] = step_of(vpar[u][i].x) * v_unit.v;
                        if (vs[u][i][1] != 0.f) vs[u][i][1] = step_of(vpar[u][i].y) * v_unit.v;
                    }
                bool all = true;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    Query& q = state[c];
                    const float top = max_keys(tops[c]);
                    const bool fresh = sum_keys(q.l) == 0.f;
                    const bool move = top > -INFINITY && (fresh || top > 7.f);
                    const float f = fresh || !move ? 1.f : ex2_approx(-top);
                    if (move) {
                        q.shift -= top;
#pragma unroll
                        for (int u = 0; u < I; ++u) y[u][c] -= top, y[u][2 + c] -= top;
                    }
                    q.l *= f;
                    q.moff[0] *= f;
                    q.moff[1] *= f;
#pragma unroll
                    for (int cb = 0; cb < 8; ++cb) out[cb][c] *= f * fv, out[cb][2 + c] *= f * fv;
                    // a column that will see a key later has no shift yet
                    all &= !fresh || move || limit[c] <= pos + 16 * I;
                }
                settled = __all_sync(0xffffffffu, all);
            }
            // weights, and with the values' steps the second product's B operand
            uint32_t pb[I][2][2];  // [64 channels][tokens 0..7, 8..15]
            auto weigh = [&](auto masked) {
#pragma unroll
                for (int u = 0; u < I; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint2 par = vpar[u][i];
                        const float m0 = fmaf(8.f, step_of(par.x), least_of(par.x));
                        const float m1 = fmaf(8.f, step_of(par.y), least_of(par.y));
                        float w[2][2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float x = y[u][2 * i + c], p = ex2_approx(x);
                            // what a column does not see has no influence on it, a
                            // step or minimum that is NaN included
                            const bool none = decltype(masked)::value && x == -INFINITY;
                            state[c].l += p;
                            state[c].moff[0] = fmaf(p, none ? 0.f : m0, state[c].moff[0]);
                            state[c].moff[1] = fmaf(p, none ? 0.f : m1, state[c].moff[1]);
                            w[c][0] = p * (none ? 0.f : vs[u][i][0]);
                            w[c][1] = p * (none ? 0.f : vs[u][i][1]);
                        }
                        pb[u][0][i] = transpose8(narrow2<true>(w[0][0], w[1][0]));
                        pb[u][1][i] = transpose8(narrow2<true>(w[0][1], w[1][1]));
                    }
            };
            if (edge) weigh(Bool<true>{});
            else weigh(Bool<false>{});
#pragma unroll
            for (int u = 0; u < I; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 x =
                        reinterpret_cast<const uint4*>(base + to_v + codes_at[u])[lane + 32 * h];
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t ca[4];
                        centred_codes(w[k], ca[0], ca[1], ca[2], ca[3]);
                        mma_f16(out[4 * h + k], ca, pb[u][h][0], pb[u][h][1]);
                    }
                }
        }
        // the stage's last fields are read before it is given back
        const bool end = flags & kEnd;
        Stage st;
        if (end) st = sh.stage[stage];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[stage]);
        if (++stage == kStages) stage = 0, phase ^= 1;
        if (!end) continue;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            Query& q = state[c];
            q.l = sum_keys(q.l);
            q.moff[0] = sum_keys(q.moff[0]);
            q.moff[1] = sum_keys(q.moff[1]);
            if (g == 0) sh.stat[warp][2 * t + c] = make_float2(q.shift, q.l);
        }
        finish_segment<F16>(a, sh, st, [&](float (*sums)[kPad], auto add) {
            constexpr bool kAdd = decltype(add)::value;
            const float back = pow2(-exponent(v_unit.v)), low = kLow * back, high = kHigh * back;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float f = warp_factor(sh, 2 * t + c, state[c]);
                float* dst = sums[2 * t + c] + g;
                const float m[2] = {state[c].moff[0] * f, state[c].moff[1] * f};
                const bool none = state[c].l == 0.f;
#pragma unroll
                for (int cb = 0; cb < 8; ++cb) {
                    const float x = none ? 0.f : fmaf(out[cb][c], low * f, m[cb >> 2]);
                    const float z = none ? 0.f : fmaf(out[cb][2 + c], high * f, m[cb >> 2]);
                    dst[16 * cb] = kAdd ? dst[16 * cb] + x : x;
                    dst[16 * cb + 8] = kAdd ? dst[16 * cb + 8] + z : z;
                }
            }
        });
        reset();
    }
}

// Sixteen queries, the rows g and g + 8; keys, and then value channels, are the
// eight columns of two products: the same words of codes are B operands here,
// keys 0..7 and 8..15 (or channels) of the low and the high four bits.  A lane's
// scores are keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9, which as they are make the A
// operand of the second product.
template <bool F16>
__device__ __forceinline__ void attend_wide(const DecodeArgs& a, Shared<true>& sh,
                                            const uint8_t* sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int to_v = part_bytes(piece_tokens(a));
    int stage = 0, len = 0;
    uint32_t phase = 0;
    float out[16][4];  // channels 8 n + 2 t + e
    Query state[2];
    Unit v_unit;
    bool settled;
    auto reset = [&] {
        settled = false;
        v_unit = {};
        state[0] = state[1] = {};
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[n][i] = 0.f;
    };
    reset();
    // over the four lanes that hold the other keys of the same queries
    auto max4 = [](float x) {
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
    };
    auto sum4 = [](float x) {
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        return x + __shfl_xor_sync(0xffffffffu, x, 2);
    };
    for (;;) {
        if (!wait_warp(sh, &sh.full[stage], phase)) return;
        const uint32_t flags = sh.stage[stage].flags;
        if (flags & kNoMore) return;
        if (flags & kStart) {
            const Stage st = sh.stage[stage];
            len = st.len;
            load_queries<F16>(a, sh, st);
        }
#pragma unroll 1
        for (int mine = 2 * warp; mine < 2 * warp + 2; ++mine) {
            if (!(flags >> mine & 1)) continue;
            // (queries are read again for each group, not kept)
            asm volatile("" ::: "memory");
            const int pos = sh.stage[stage].pos + 16 * mine;
            const uint8_t* base = sm + stage * kStageBytes;
            int codes_at, pars_at;
            group_places(a, mine, codes_at, pars_at);
            float y[2][4];  // [keys 0..7, 8..15][2 i + e]
            {
                float acc[2][2][4] = {};  // [keys][64 channels]
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    asm volatile("" ::: "memory");  // (nor all of them at once)
                    const uint4 x = reinterpret_cast<const uint4*>(base + codes_at)[lane + 32 * h];
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 q4 = *reinterpret_cast<const uint4*>(sh.q[4 * h + k][lane]);
                        const uint32_t qa[4] = {q4.x, q4.y, q4.z, q4.w};
                        uint32_t lo0, hi0, lo1, hi1;
                        codes(w[k], lo0, hi0, lo1, hi1);
                        mma_f16(acc[0][h], qa, lo0, hi0);
                        mma_f16(acc[1][h], qa, lo1, hi1);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // of keys 8 j + 2 t and the next
                    const uint4 par = *reinterpret_cast<const uint4*>(base + pars_at +
                                                                      (8 * j + 2 * t) * 8);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t p0 = e ? par.z : par.x, p1 = e ? par.w : par.y;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 qs = sh.qsum[g + 8 * i];
                            float d = least_of(p0) * qs.x;
                            d = fmaf(least_of(p1), qs.y, d);
                            d = fmaf(step_of(p0), acc[j][0][2 * i + e], d);
                            d = fmaf(step_of(p1), acc[j][1][2 * i + e], d);
                            y[j][2 * i + e] = fmaf(d, sh.unit[g + 8 * i], state[i].shift);
                        }
                    }
                }
            }
            const bool edge =
                pos > len - a.krows + 1 - 16 || (a.window && pos < len - a.window);
            if (edge) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int hi = sh.limit[g + 8 * i], lo = a.window ? max(0, hi - a.window) : 0;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int at = pos + 8 * j + 2 * t + e;
                            if (at < lo || at >= hi) y[j][2 * i + e] = -INFINITY;
                        }
                }
            }
            uint4 vpar[2];
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                vpar[j] = *reinterpret_cast<const uint4*>(base + to_v + pars_at +
                                                          (8 * j + 2 * t) * 8);
                if (edge) {  // whatever the cache holds behind a sequence's end
                    const int at = pos + 8 * j + 2 * t;
                    if (at >= len) vpar[j].x = vpar[j].y = 0u;
                    if (at + 1 >= len) vpar[j].z = vpar[j].w = 0u;
                }
                most = fmaxf(most, fmaxf(fmaxf(step_of(vpar[j].x), step_of(vpar[j].y)),
                                         fmaxf(step_of(vpar[j].z), step_of(vpar[j].w))));
            }
            float tops[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                tops[i] = fmaxf(fmaxf(y[0][2 * i], y[0][2 * i + 1]),
                                fmaxf(y[1][2 * i], y[1][2 * i + 1]));
            if (__any_sync(0xffffffffu, !settled || most * v_unit.v >= 256.f || tops[0] > 7.f ||
                                            tops[1] > 7.f)) {
                // (all lanes agree on the unit: the steps of a group are theirs together)
                const float fv = v_unit.fit(max4(most));
                bool all = true;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    Query& q = state[i];
                    const float top = max4(tops[i]);
                    const bool fresh = sum4(q.l) == 0.f;
                    const bool move = top > -INFINITY && (fresh || top > 7.f);
                    const float f = fresh || !move ? 1.f : ex2_approx(-top);
                    if (move) {
                        q.shift -= top;
#pragma unroll
                        for (int j = 0; j < 2; ++j) y[j][2 * i] -= top, y[j][2 * i + 1] -= top;
                    }
                    q.l *= f;
                    q.moff[0] *= f;
                    q.moff[1] *= f;
                    const float both = f * fv;
                    if (__any_sync(0xffffffffu, both != 1.f))
#pragma unroll
                        for (int n = 0; n < 16; ++n)
                            out[n][2 * i] *= both, out[n][2 * i + 1] *= both;
                    all &= !fresh || move || sh.limit[g + 8 * i] - 16 <= pos;
                }
                settled = __all_sync(0xffffffffu, all);
            }
            uint32_t pa[2][4];  // [64 channels]: the A operand
            auto weigh = [&](auto masked) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float w[2][2][2];  // [i][e][64 channels]
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t p0 = e ? vpar[j].z : vpar[j].x;
                        const uint32_t p1 = e ? vpar[j].w : vpar[j].y;
                        const float m0 = fmaf(8.f, step_of(p0), least_of(p0));
                        const float m1 = fmaf(8.f, step_of(p1), least_of(p1));
                        const float s0 = step_of(p0) * v_unit.v, s1 = step_of(p1) * v_unit.v;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float x = y[j][2 * i + e], p = ex2_approx(x);
                            const bool none = decltype(masked)::value && x == -INFINITY;
                            state[i].l += p;
                            state[i].moff[0] = fmaf(p, none ? 0.f : m0, state[i].moff[0]);
                            state[i].moff[1] = fmaf(p, none ? 0.f : m1, state[i].moff[1]);
                            w[i][e][0] = p * (none ? 0.f : s0);
                            w[i][e][1] = p * (none ? 0.f : s1);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            pa[h][2 * j + i] = narrow2<true>(w[i][0][h], w[i][1][h]);
                }
            };
            if (edge) weigh(Bool<true>{});
            else weigh(Bool<false>{});
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 x =
                    reinterpret_cast<const uint4*>(base + to_v + codes_at)[lane + 32 * h];
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t lo0, hi0, lo1, hi1;
                    centred_codes(w[k], lo0, hi0, lo1, hi1);
                    mma_f16(out[8 * h + 2 * k], pa[h], lo0, lo1);
                    mma_f16(out[8 * h + 2 * k + 1], pa[h], hi0, hi1);
                }
            }
        }
        const bool end = flags & kEnd;
        Stage st;
        if (end) st = sh.stage[stage];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[stage]);
        if (++stage == kStages) stage = 0, phase ^= 1;
        if (!end) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            Query& q = state[i];
            q.l = sum4(q.l);
            q.moff[0] = sum4(q.moff[0]);
            q.moff[1] = sum4(q.moff[1]);
            if (t == 0) sh.stat[warp][g + 8 * i] = make_float2(q.shift, q.l);
        }
        finish_segment<F16>(a, sh, st, [&](float (*sums)[kPad], auto add) {
            constexpr bool kAdd = decltype(add)::value;
            const float back = pow2(-exponent(v_unit.v)), low = kLow * back, high = kHigh * back;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float f = warp_factor(sh, g + 8 * i, state[i]);
                float* dst = sums[g + 8 * i] + 2 * t;
                const float m[2] = {state[i].moff[0] * f, state[i].moff[1] * f};
                const bool none = state[i].l == 0.f;
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    const float unit = (n & 1 ? high : low) * f;
                    float2 x = make_float2(fmaf(out[n][2 * i], unit, m[n >> 3]),
                                           fmaf(out[n][2 * i + 1], unit, m[n >> 3]));
                    if (none) x = make_float2(0.f, 0.f);
                    float2* at = reinterpret_cast<float2*>(dst + 8 * n);
                    *at = kAdd ? add2(*at, x) : x;
                }
            }
        });
        reset();
    }
}

template <bool F16, bool WIDE>
__global__ void __launch_bounds__(kThreads, kCtas) attn_decode_kernel(DecodeArgs a) {
    extern __shared__ __align__(128) uint8_t sm[];
    Shared<WIDE>& sh = *reinterpret_cast<Shared<WIDE>*>(sm + kStages * kStageBytes);
    if (threadIdx.x == 0) {
        sh.stop = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_release();
    if (threadIdx.x >= kWarps * 32) copy_role(a, sh, sm);
    else if constexpr (WIDE) attend_wide<F16>(a, sh, sm);
    else attend_narrow<F16>(a, sh, sm);
}

// Joins what several CTAs have of one (sequence, head, block).  CTA (x, y) has
// job x and of its queries every gridDim.y-th, `per` of them; each has 8 / per
// warps, which share the pieces, four channels a lane.  What there is to do the
// main kernel has written down (found here from all lengths, a CTA for every
// (sequence, head, block), 64 sequences of 2000 to 8192 tokens took 92.9 us where
// this takes 89.8, one of 777 12.5, and this 11.6).
constexpr int kJoinWarps = 8;  // (16: 84.5 us where 8 take 83.4, at 64 sequences)
template <bool F16, bool WIDE>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join_kernel(DecodeArgs a) {
    constexpr int Q = kRows<WIDE>;
    __shared__ float4 parts[kJoinWarps][32];
    __shared__ float part_sum[kJoinWarps], part_least[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const int4 j = __ldcg(reinterpret_cast<const int4*>(a.jobs + blockIdx.x));
    const int n = j.x, b0 = j.z, b1 = j.w;
    if (b1 <= b0) return;
    // (a main kernel that gave up may have left anything)
    if (b0 < 0 || b1 >= a.pieces || n < 0 || n >= a.n_seqs || j.y < 0 ||
        j.y >= a.c.kv_heads * a.blocks)
        return;
    const int head = j.y / a.blocks, block = j.y - head * a.blocks;
    const float2* stat = reinterpret_cast<const float2*>(a.part + 2LL * a.pieces * Q * D);
    const int per = Q / gridDim.y, shares = kJoinWarps / per;  // powers of two
    const int mine = warp / shares, share = warp - mine * shares;
    const int c = blockIdx.y + mine * gridDim.y, row = block * Q + c;
    // this warp's pieces: their least shift, then everything brought to it
    float least = INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int from = b0 + share; from <= b1; from += 32 * shares) {
        const int b = from + lane * shares;
        float2 s = make_float2(0.f, 0.f);
        if (b <= b1) s = __ldcg(stat + (2 * b + (b == b0)) * Q + c);
        float low = s.y != 0.f ? s.x : INFINITY;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1)
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, off));
        if (low < least) {
            const float f = least < INFINITY ? ex2_approx(low - least) : 0.f;
            o.x *= f, o.y *= f, o.z *= f, o.w *= f, sum *= f;
            least = low;
        }
        const float f = s.y != 0.f ? ex2_approx(least - s.x) : 0.f;
        sum = s.y != 0.f ? fmaf(s.y, f, sum) : sum;
        const int here = min(32, (b1 - from) / shares + 1);
#pragma unroll 8
        for (int i = 0; i < here; ++i) {
            const int bi = from + i * shares, slot = 2 * bi + (bi == b0);
            const float4 x = __ldcg(
                reinterpret_cast<const float4*>(a.part + ((long long)slot * Q + c) * D) + lane);
            const float fi = __shfl_sync(0xffffffffu, f, i);
            if (fi == 0.f) continue;
            o.x = fmaf(x.x, fi, o.x);
            o.y = fmaf(x.y, fi, o.y);
            o.z = fmaf(x.z, fi, o.z);
            o.w = fmaf(x.w, fi, o.w);
        }
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (shares > 1) {
        parts[warp][lane] = o;
        if (lane == 0) part_sum[warp] = sum, part_least[warp] = least;
        __syncthreads();
        if (share) return;
        float all = INFINITY;
        for (int w = warp; w < warp + shares; ++w) all = fminf(all, part_least[w]);
        o = make_float4(0.f, 0.f, 0.f, 0.f);
        sum = 0.f;
        for (int w = warp; w < warp + shares; ++w) {
            if (!(part_least[w] < INFINITY)) continue;
            const float f = ex2_approx(all - part_least[w]);
            const float4 x = parts[w][lane];
            o.x = fmaf(x.x, f, o.x);
            o.y = fmaf(x.y, f, o.y);
            o.z = fmaf(x.z, f, o.z);
            o.w = fmaf(x.w, f, o.w);
            sum = fmaf(part_sum[w], f, sum);
        }
        least = all;
    }
    if (row >= a.rows) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int i_row = row / a.group;
    const long long at = ((long long)n * a.krows + i_row) * a.heads + head * a.group + row -
                         i_row * a.group;
    reinterpret_cast<uint2*>(a.o + at * D)[lane] =
        make_uint2(narrow2<F16>(o.x * inv, o.y * inv), narrow2<F16>(o.z * inv, o.w * inv));
    if (a.lse && lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : (log2f(sum) - least) * kLn2;
}

// Query columns of a block: 8 where that is all, else 16.
inline int columns(int rows) { return rows <= 8 ? 8 : 16; }

template <bool F16, bool WIDE>
cudaError_t launch(const DecodeArgs& a, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<F16, WIDE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes<WIDE>());
    if (e != cudaSuccess) return e;
    launch_pdl(attn_decode_kernel<F16, WIDE>, dim3(a.pieces), dim3(kThreads), smem_bytes<WIDE>(), s, a);
    // few units: their queries to CTAs of their own
    const long long units = (long long)a.n_seqs * a.c.kv_heads * a.blocks;
    int apart = kRows<WIDE> / kJoinWarps;
    while (apart < kRows<WIDE> && 2 * apart * units <= 304) apart *= 2;
    const unsigned jobs = (unsigned)std::min<long long>(units, a.pieces);
    return launch_pdl(attn_join_kernel<F16, WIDE>, dim3(jobs, apart),
                      dim3(kJoinWarps * 32), 0, s, a);
}

}  // namespace

cudaError_t status_word_decode(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_decode_status);
}

}  // namespace kda

using namespace kda;

// Two incomplete segments per piece; the call makes no more pieces than
// KDA_KV4_PIECES (three CTAs on each of 160 multiprocessors).
extern "C" size_t kda_attn_kv4_workspace_size(int n_seqs, int krows, int heads, int kv_heads) {
    if (n_seqs < 1 || krows < 1 || krows > KDA_MAX_K || heads < 1 || kv_heads < 1 ||
        heads % kv_heads)
        return 0;
    const size_t q = (size_t)columns(krows * (heads / kv_heads));
    return KDA_KV4_PIECES * (2 * q * (D + 2) * sizeof(float) + sizeof(Job));
}

extern "C" kda_status kda_attn_kv4_decode(const void* q, const uint8_t* cache, int64_t n_pages,
                                          int page, const int* page_table, int max_pages,
                                          const int* lens, void* o, float* lse, int n_seqs,
                                          int krows, int heads, int kv_heads, int head_dim,
                                          int in_dtype, int window, float scale, void* workspace,
                                          size_t workspace_bytes, uint64_t stream) {
    const char* fn = "kda_attn_kv4_decode";
    KDA_REQUIRE(in_dtype == KDA_F32 || in_dtype == KDA_BF16 || in_dtype == KDA_F16,
                KDA_ERR_INVALID_ARG, "%s: in_dtype %d is not a kda_dtype", fn, in_dtype);
    KDA_REQUIRE(in_dtype != KDA_F32, KDA_ERR_UNSUPPORTED, "%s: FP32 rows are not built", fn);
    kda_status st = validate_cache(fn, cache, n_pages, page, page_table, max_pages, lens, n_seqs,
                                   kv_heads, head_dim);
    if (st != KDA_OK) return st;
    KDA_REQUIRE(krows >= 1 && krows <= KDA_MAX_K, KDA_ERR_INVALID_ARG,
                "%s: krows (%d) must be in 1..%d", fn, krows, KDA_MAX_K);
    KDA_REQUIRE(heads >= 1 && heads % kv_heads == 0, KDA_ERR_INVALID_ARG,
                "%s: heads (%d) must be a positive multiple of kv_heads (%d)", fn, heads,
                kv_heads);
    KDA_REQUIRE(window >= 0, KDA_ERR_INVALID_ARG, "%s: window (%d) must be >= 0", fn, window);
    KDA_REQUIRE(std::isfinite(scale) && scale > 0.f, KDA_ERR_INVALID_ARG,
                "%s: scale must be finite and positive", fn);
    st = validate_rows(fn, "q", q, (int64_t)heads * D, heads);
    if (st == KDA_OK) st = validate_rows(fn, "o", o, (int64_t)heads * D, heads);
    if (st != KDA_OK) return st;
    const int group = heads / kv_heads, rows = krows * group, cols = columns(rows);
    const int blocks = (rows + cols - 1) / cols;
    KDA_REQUIRE((long long)n_seqs * kv_heads * blocks < 0x7fffffffLL, KDA_ERR_INVALID_ARG,
                "%s: problem too large", fn);
    const size_t need = kda_attn_kv4_workspace_size(n_seqs, krows, heads, kv_heads);
    KDA_REQUIRE(workspace && workspace_bytes >= need, KDA_ERR_WORKSPACE,
                "%s: workspace of %zu B, %zu B needed", fn, workspace ? workspace_bytes : 0, need);
    KDA_REQUIRE(aligned16(workspace), KDA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned",
                fn);
    KDA_REQUIRE(!fault_injected(), KDA_ERR_CUDA, "%s: injected launch failure", fn);
    const int ctas = kCtas * sm_count();
    const int pieces = ctas < KDA_KV4_PIECES ? ctas : KDA_KV4_PIECES;
    KDA_REQUIRE(pieces > 0, KDA_ERR_CUDA, "%s: no device", fn);
    const int reach = (int)(window ? std::min(0x7fffffffLL, (long long)window + krows - 1)
                                   : 0x7fffffffLL);
    DecodeArgs a = {(const uint16_t*)q, (uint16_t*)o, lse, n_seqs, krows, heads, window, reach,
                    group, rows, blocks, scale, pieces, static_cast<float*>(workspace),
                    reinterpret_cast<Job*>(static_cast<float*>(workspace) +
                                           (size_t)KDA_KV4_PIECES * 2 * cols * (D + 2)),
                    {const_cast<uint8_t*>(cache), page_table, lens, n_pages, max_pages,
                     __builtin_ctz((unsigned)page), kv_heads}};
    cudaStream_t s = as_stream(stream);
    const bool f16 = in_dtype == KDA_F16;
    cudaError_t e;
    if (cols == 8) e = f16 ? launch<true, false>(a, s) : launch<false, false>(a, s);
    else e = f16 ? launch<true, true>(a, s) : launch<false, true>(a, s);
    if (e != cudaSuccess) {
        set_error("%s: launch failed: %s", fn, cudaGetErrorString(e));
        return KDA_ERR_CUDA;
    }
    return launch_result(fn);
}
