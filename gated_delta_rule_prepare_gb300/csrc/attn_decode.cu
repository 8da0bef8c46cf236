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
//  - The cache keeps codes in the order of mma.sync's A operand: keys (or value
//    channels) are the product's 16 rows, queries its 8 columns, so that one
//    query row in use wastes 7 of 8 columns of an instruction that is not the
//    bound, and no shared-memory transposition is needed.
//  - A score's columns are queries, as an output's are: running sums and
//    rescaling stay within a lane.  p_t s_ta is rounded to FP16 after a common
//    power of two that keeps it below 2^15 (11 significant bits; weights down to
//    2^-33 of the largest); scores, sums and outputs are FP32.
//
// All positions of the batch, in chunks of 128 tokens, are one line that the
// CTAs cut into equal pieces, whatever the lengths: a piece ends where it ends,
// and what is left of a (sequence, head) in each is joined by a second kernel
// (attn_join_kernel), always in the same order.  Per CTA one warp copies chunks
// into a ring in shared memory and four attend over them.
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

// A chunk is 8 groups of 16 tokens; each of a CTA's four warps takes two: with 8
// query columns together, so that their products and weights run in each other's
// waits, with 16 one after the other.  Several small CTAs to a multiprocessor,
// not one large one: while one ends a segment the others go on.  The registers
// that leaves a thread hold all it has; what spills costs more than anything else
// here, as the rings leave next to no L1 cache.
constexpr int kWarps = 4;  // and one that copies
constexpr int kThreads = (kWarps + 1) * 32;
template <int NT>
constexpr int kCtas = NT == 1 ? 3 : 2;
template <int NT>
constexpr int kStages = NT == 1 ? 3 : 4;
template <int NT>
constexpr int kIlp = NT == 1 ? 2 : 1;
constexpr int kGroups = 8;
constexpr int kChunk = kGroups * 16;  // tokens
constexpr int kStageBytes = kChunk * kTokenBytes;

struct DecodeArgs {
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    int n_seqs, krows, heads, window;
    int group, rows, blocks;  // heads per KV head; query rows of a KV head; blocks of them
    float scale;
    int pieces;  // CTAs of the main kernel
    float* part;  // [2 * pieces][8 * NT][128] sums, then [2 * pieces][8 * NT] (shift, l)
    Cache c;
};

// Chunks that sequence n's queries see: [first, first + count).
struct Chunks {
    int first, count;
};
__device__ __forceinline__ int good_len(const DecodeArgs& a, int len) {
    return len < 0 || (long long)len > ((long long)a.c.max_pages << a.c.page_shift) ? 0 : len;
}
__device__ __forceinline__ Chunks chunks_of(const DecodeArgs& a, int len) {
    const int lo = (a.window ? max(0, len - a.krows - a.window + 1) : 0) / kChunk;
    return {lo, len > 0 ? (len - 1) / kChunk + 1 - lo : 0};
}
// The line of `total` chunks in pieces, none of them empty: their number, and
// where piece b starts.
__device__ __forceinline__ int piece_count(const DecodeArgs& a, long long total) {
    return (int)min((long long)a.pieces, total);
}
__device__ __forceinline__ long long piece_start(const DecodeArgs& a, long long total, int b) {
    const int pieces = piece_count(a, total);
    return b >= pieces ? total : total * b / pieces;
}

// All lengths by one warp: the chunks of all sequences of one (head, block),
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
            const int mine = chunks_of(a, good_len(a, len[i])).count;
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
// (sequence, head, block of 8 NT query rows).
struct Stage {
    int pos;         // the chunk's first position
    uint32_t flags;  // bit i: tokens 16 i .. 16 i + 15 are in the stage; then:
    int len;         // of the sequence
    int n, head, block;
    int part;  // where an incomplete segment's sums go, or -1
};
constexpr uint32_t kStart = 1u << 24, kEnd = 1u << 25, kNoMore = 1u << 26;

constexpr int kPad = 132;  // a query's 128 sums, so that a warp's stores meet all banks
template <int NT>
struct Shared {
    uint64_t full[kStages<NT>], empty[kStages<NT>];
    Stage stage[kStages<NT>];
    // the segment's queries as B operands (FP16, scaled by a power of two); by
    // query, the factor from a product to a score in log2 units and the sums
    // over 64 channels
    uint2 q[NT][8][32];
    float unit[8 * NT];
    float2 qsum[8 * NT];
    // its end
    float2 stat[kWarps][8 * NT];  // a warp's (shift, l) by query
    float factor[kWarps][8 * NT];
    float2 joint[8 * NT];
    float4 sums[2][8 * NT][kPad / 4];  // two warps' outputs at a time
    int stop;
};
template <int NT>
constexpr int smem_bytes() {
    return kStages<NT> * kStageBytes + (int)sizeof(Shared<NT>);
}

template <bool B>
struct Bool {
    static constexpr bool value = B;
};

// Waits end: with the phase, with another role's giving up, or after 2^33 clocks.
template <int NT>
__device__ __forceinline__ bool wait_warp(Shared<NT>& sh, uint64_t* bar, uint32_t parity) {
    bool ok = mbar_wait(bar, parity, 1);
    if (!ok) {
        const long long from = clock64();
        while (!(ok = mbar_wait(bar, parity, 32))) {
            if (*(volatile int*)&sh.stop) break;
            if (clock64() - from > 1LL << 33) {
                atomicOr(&g_decode_status, STATUS_TIMEOUT);
                *(volatile int*)&sh.stop = 1;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// Tokens that lie together in the cache and in a stage: a stage holds pieces of
// so many, each laid out as a page of its size, so that a page of up to 128
// tokens is one copy.  (Small copies cost what large ones do: with four to a
// page, codes and parameters apart, copying alone took 75 us where it takes
// COPYUS, 64 sequences of 2000 to 8192 tokens.)
__device__ __forceinline__ int piece_tokens(const DecodeArgs& a) { return min(a.c.page(), 128); }

// The copying warp: walks this CTA's piece of the line.
template <int NT>
__device__ __forceinline__ void copy_role(const DecodeArgs& a, Shared<NT>& sh, uint8_t* sm) {
    const int lane = threadIdx.x & 31;
    const int heads = a.c.kv_heads, per_seq = heads * a.blocks;
    bool bad_len = false;
    const long long one = scan_lengths(a, [](int, long long, int) { return true; });
    const long long total = one * per_seq;
    const long long from = piece_start(a, total, blockIdx.x);
    const long long to = piece_start(a, total, blockIdx.x + 1);
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
        // (n, head, block) units of this sequence, chunk by chunk
        while (go && at < to && at < n_start + (long long)ch.count * per_seq) {
            const int unit = (int)((at - n_start) / ch.count);
            const int head = unit / a.blocks, block = unit - head * a.blocks;
            const long long u_start = n_start + (long long)unit * ch.count;
            const long long u_end = u_start + ch.count;
            const long long seg_end = min(u_end, to);
            const bool whole = at == u_start && seg_end == u_end;
            const int part = whole ? -1 : 2 * (int)blockIdx.x + (at == from ? 0 : 1);
            const long long seg_start = at;
            const int* table = a.c.table + (long long)n * a.c.max_pages;
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
                if (++stage == kStages<NT>) stage = 0, phase ^= 1;
            }
        }
        n_start += (long long)ch.count * per_seq;
        ++n;
    }
    if (go) go = wait_warp(sh, &sh.empty[stage], phase ^ 1);
    if (lane == 0) {
        if (go) {
            sh.stage[stage].flags = kNoMore;
            mbar_arrive(&sh.full[stage]);
        } else {
            // copies in flight land before the CTA's memory goes away
            for (int s = 0; s < kStages<NT>; ++s)
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

template <bool F16, int NT>
__device__ __forceinline__ void attend_role(const DecodeArgs& a, Shared<NT>& sh,
                                            const uint8_t* sm) {
    constexpr int Q = 8 * NT;  // query columns
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    constexpr int I = kIlp<NT>;
    // where this warp's groups of a stage are: codes, parameters, of K; of V by
    // `to_v` further
    constexpr int N = kGroups / kWarps;
    int codes_at[N], pars_at[N];
    const int to_v = part_bytes(piece_tokens(a));
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int tok = (N * warp + u) * 16, piece = piece_tokens(a);
        const int in = tok & (piece - 1), block = (tok - in) * kTokenBytes;
        codes_at[u] = block + in * 64;
        pars_at[u] = block + piece * 64 + in * 8;
    }
    int stage = 0;
    uint32_t phase = 0;
    // with 8 query columns in registers, with 16 read again for each group
    uint2 qb[NT == 1 ? 8 : 1];
    float unit[NT == 1 ? 2 : 1], qsum[NT == 1 ? 2 : 1][2];
    (void)qb, (void)unit, (void)qsum;
    int len = 0;
    float out[NT][8][4];
    // weights are 2^(score + shift), at most 2^7; l sums them, moff weights times
    // m + 8 s, by 64 channels; steps enter times v_unit, below 2^8 then
    float shift[NT][2], l[NT][2], moff[NT][2][2], v_unit = 1.f;
    bool settled = false;  // every column has a shift that comes from a score
    auto limit_of = [&](int block, int nt, int c) {  // positions from it on are not seen
        const int row = block * Q + nt * 8 + 2 * t + c;
        return row < a.rows ? len - a.krows + row / a.group + 1 : 0;
    };
    for (;;) {
        if (!wait_warp(sh, &sh.full[stage], phase)) return;
        const uint32_t flags = sh.stage[stage].flags;
        if (flags & kNoMore) return;
        if (flags & kStart) {
            const Stage st = sh.stage[stage];
            len = st.len;
            settled = false;
#pragma unroll 1
            for (int r = warp; r < Q; r += kWarps) {  // a query row, four channels a lane
                const int row = st.block * Q + r;
                const int i = row / a.group, hh = row - i * a.group;
                uint2 raw = make_uint2(0u, 0u);
                if (row < a.rows)
                    raw = __ldg(reinterpret_cast<const uint2*>(
                                    a.q + (((long long)st.n * a.krows + i) * a.heads +
                                           st.head * a.group + hh) * D) + lane);
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
                for (int off = 1; off < 16; off <<= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, off);
                // channel 16 kb + 8 j + 2 t + e: codes of j = 1 are the high four bits
                const int kb = lane >> 2, j = lane >> 1 & 1, t0 = 2 * (lane & 1);
                const float fj = j ? kHigh / kLow : 1.f;
                uint32_t* dst = reinterpret_cast<uint32_t*>(&sh.q[r >> 3][kb][(r & 7) * 4 + t0]);
                dst[j] = narrow2<true>(x.x * fj, x.y * fj);
                dst[2 + j] = narrow2<true>(y.x * fj, y.y * fj);
                if (lane == 0) {
                    sh.unit[r] = a.scale * kLog2e * kLow * pow2(-up);
                    sh.qsum[r].x = sum * (1.f / kLow);
                }
                if (lane == 16) sh.qsum[r].y = sum * (1.f / kLow);
            }
            consumer_sync();
            if constexpr (NT == 1) {
#pragma unroll
                for (int k = 0; k < 8; ++k) qb[k] = sh.q[0][k][lane];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    unit[c] = sh.unit[2 * t + c];
                    qsum[c][0] = sh.qsum[2 * t + c].x;
                    qsum[c][1] = sh.qsum[2 * t + c].y;
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    shift[nt][c] = l[nt][c] = moff[nt][c][0] = moff[nt][c][1] = 0.f;
#pragma unroll
                for (int cb = 0; cb < 8; ++cb)
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) out[nt][cb][i4] = 0.f;
            }
        }
#pragma unroll 1
        for (int first = 0; first < N; first += I) {
            const int mine = N * warp + first;
            // a group that is not there, behind one that is: its tokens are masked
            if (!(flags >> mine & ((1u << I) - 1))) continue;
            // (queries are read again for each group, not kept)
            asm volatile("" ::: "memory");
            const int pos = sh.stage[stage].pos + 16 * mine;
            int ca_at[I], pa_at[I];
#pragma unroll
            for (int u = 0; u < I; ++u) {
                ca_at[u] = codes_at[u];
                pa_at[u] = pars_at[u];
#pragma unroll
                for (int x = 1; x < N; ++x)
                    if (I == 1 && first == x) ca_at[u] = codes_at[x], pa_at[u] = pars_at[x];
            }
            const uint8_t* base = sm + stage * kStageBytes;
            // scores of tokens g and g + 8 of each group
            float y[I][NT][4];
            {
                float acc[I][NT][2][4] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int u = 0; u < I; ++u) {
                        const uint4 x = reinterpret_cast<const uint4*>(
                            base + ca_at[u])[lane + 32 * h];
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t ca[4];
                            codes(w[k], ca[0], ca[2], ca[1], ca[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint2 b =
                                    NT == 1 ? qb[4 * h + k] : sh.q[nt][4 * h + k][lane];
                                mma_f16(acc[u][nt][h], ca, b.x, b.y);
                            }
                        }
                    }
#pragma unroll
                for (int u = 0; u < I; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint2 par = reinterpret_cast<const uint2*>(
                            base + pa_at[u])[g + 8 * i];
                        const float sa = __uint_as_float(par.x << 16);
                        const float ma = __uint_as_float(par.x & 0xffff0000u);
                        const float sb = __uint_as_float(par.y << 16);
                        const float mb = __uint_as_float(par.y & 0xffff0000u);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float un, q0, q1;
                                if constexpr (NT == 1) {
                                    un = unit[c], q0 = qsum[c][0], q1 = qsum[c][1];
                                } else {
                                    const float2 qs = sh.qsum[8 * nt + 2 * t + c];
                                    un = sh.unit[8 * nt + 2 * t + c], q0 = qs.x, q1 = qs.y;
                                }
                                float d = ma * q0;
                                d = fmaf(mb, q1, d);
                                d = fmaf(sa, acc[u][nt][0][2 * i + c], d);
                                d = fmaf(sb, acc[u][nt][1][2 * i + c], d);
                                y[u][nt][2 * i + c] = fmaf(d, un, shift[nt][c]);
                            }
                    }
            }
            const bool edge = pos + 16 * I > len - a.krows + 1 ||
                              (a.window && pos < len - a.window) ||
                              (flags >> mine & ((1u << I) - 1)) != (1u << I) - 1;
            if (edge) {
                const int block = sh.stage[stage].block;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int hi = limit_of(block, nt, c);
                        const int lo = a.window ? max(0, hi - a.window) : 0;
#pragma unroll
                        for (int u = 0; u < I; ++u)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int at = pos + 16 * u + g + 8 * i;
                                if (at < lo || at >= hi || !(flags >> (mine + u) & 1))
                                    y[u][nt][2 * i + c] = -INFINITY;
                            }
                    }
            }
            uint2 vpar[I][2];
            float vs[I][2][2], most = 0.f;
#pragma unroll
            for (int u = 0; u < I; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    vpar[u][i] = reinterpret_cast<const uint2*>(
                        base + to_v + pa_at[u])[g + 8 * i];
                    vs[u][i][0] = __uint_as_float(vpar[u][i].x << 16) * v_unit;
                    vs[u][i][1] = __uint_as_float(vpar[u][i].y << 16) * v_unit;
                    // whatever the cache holds behind a sequence's end
                    if (edge && (pos + 16 * u + g + 8 * i >= len || !(flags >> (mine + u) & 1)))
                        vs[u][i][0] = vs[u][i][1] = 0.f;
                    most = fmaxf(most, fmaxf(vs[u][i][0], vs[u][i][1]));
                }
            bool over = !settled || most >= 256.f;
            float tops[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    tops[nt][c] = fmaxf(y[0][nt][c], y[0][nt][2 + c]);
#pragma unroll
                    for (int u = 1; u < I; ++u)
                        tops[nt][c] = fmaxf(fmaxf(tops[nt][c], y[u][nt][c]), y[u][nt][2 + c]);
                    over |= tops[nt][c] > 7.f;
                }
            if (__any_sync(0xffffffffu, over)) {
                // shifts: from the first scores of a column, and again once a
                // weight would pass 2^7; the steps' unit likewise
                most = max_keys(most);
                float fv = 1.f;
                if (most > 0.f && most < INFINITY && (!settled || most >= 256.f)) {
                    const int was = exponent(v_unit);
                    const int now = max(-126, min(126, was + 6 - exponent(most)));
                    v_unit = pow2(now);
                    fv = pow2(max(-126, min(126, now - was)));
#pragma unroll
                    for (int u = 0; u < I; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            vs[u][i][0] *= fv;
                            vs[u][i][1] *= fv;
                        }
                }
                bool all = true;
                const int block = sh.stage[stage].block;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float top = max_keys(tops[nt][c]);
                        const bool fresh = sum_keys(l[nt][c]) == 0.f;
                        const bool move = top > -INFINITY && (fresh || top > 7.f);
                        const float f = fresh || !move ? 1.f : ex2_approx(-top);
                        if (move) {
                            shift[nt][c] -= top;
#pragma unroll
                            for (int u = 0; u < I; ++u) {
                                y[u][nt][c] -= top;
                                y[u][nt][2 + c] -= top;
                            }
                        }
                        l[nt][c] *= f;
                        moff[nt][c][0] *= f;
                        moff[nt][c][1] *= f;
#pragma unroll
                        for (int cb = 0; cb < 8; ++cb) {
                            out[nt][cb][c] *= f * fv;
                            out[nt][cb][2 + c] *= f * fv;
                        }
                        // a column that will see a key later has no shift yet
                        all &= !fresh || move || limit_of(block, nt, c) <= pos + 16 * I;
                    }
                settled = __all_sync(0xffffffffu, all);
            }
            // weights, and with the values' steps the second product's B operand
            uint32_t pb[I][NT][2][2];  // [64 channels][tokens 0..7, 8..15]
            auto weigh = [&](auto masked) {
#pragma unroll
                for (int u = 0; u < I; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint2 par = vpar[u][i];
                        const float m0 = fmaf(8.f, __uint_as_float(par.x << 16),
                                              __uint_as_float(par.x & 0xffff0000u));
                        const float m1 = fmaf(8.f, __uint_as_float(par.y << 16),
                                              __uint_as_float(par.y & 0xffff0000u));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float w[2][2];
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float x = y[u][nt][2 * i + c], p = ex2_approx(x);
                                // what a column does not see has no influence on it,
                                // a step or minimum that is NaN included
                                const bool none = decltype(masked)::value && x == -INFINITY;
                                l[nt][c] += p;
                                moff[nt][c][0] = fmaf(p, none ? 0.f : m0, moff[nt][c][0]);
                                moff[nt][c][1] = fmaf(p, none ? 0.f : m1, moff[nt][c][1]);
                                w[c][0] = p * (none ? 0.f : vs[u][i][0]);
                                w[c][1] = p * (none ? 0.f : vs[u][i][1]);
                            }
                            pb[u][nt][0][i] = transpose8(narrow2<true>(w[0][0], w[1][0]));
                            pb[u][nt][1][i] = transpose8(narrow2<true>(w[0][1], w[1][1]));
                        }
                    }
            };
            if (edge) weigh(Bool<true>{});
            else weigh(Bool<false>{});
#pragma unroll
            for (int u = 0; u < I; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 x = reinterpret_cast<const uint4*>(
                        base + to_v + ca_at[u])[lane + 32 * h];
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t ca[4];
                        codes(w[k], ca[0], ca[1], ca[2], ca[3]);
                        ca[0] = sub_h2(ca[0], 0x00080008u);  // 8 * 2^-24
                        ca[1] = sub_h2(ca[1], 0x00800080u);  // 8 * 2^-20
                        ca[2] = sub_h2(ca[2], 0x00080008u);
                        ca[3] = sub_h2(ca[3], 0x00800080u);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(out[nt][4 * h + k], ca, pb[u][nt][h][0], pb[u][nt][h][1]);
                    }
                }
        }
        // the stage's last fields are read before it is given back
        const bool end = flags & kEnd;
        Stage st;
        if (end) st = sh.stage[stage];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[stage]);
        if (++stage == kStages<NT>) stage = 0, phase ^= 1;
        if (!end) continue;

        // The segment's end: the warps' sums become one.  (In short code: what
        // runs once a segment is fetched anew each time, and unrolled over a
        // thread's sums it took 7 us, with 16 columns 30.)
        const int tid = threadIdx.x;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                l[nt][c] = sum_keys(l[nt][c]);
                moff[nt][c][0] = sum_keys(moff[nt][c][0]);
                moff[nt][c][1] = sum_keys(moff[nt][c][1]);
                if (g == 0) sh.stat[warp][nt * 8 + 2 * t + c] = make_float2(shift[nt][c], l[nt][c]);
            }
        consumer_sync();
        if (tid < Q) {
            // the least shift is that of the largest score
            float least = INFINITY, sum = 0.f;
#pragma unroll 1
            for (int w = 0; w < kWarps; ++w)
                if (sh.stat[w][tid].y != 0.f) least = fminf(least, sh.stat[w][tid].x);
#pragma unroll 1
            for (int w = 0; w < kWarps; ++w) {
                const float2 x = sh.stat[w][tid];
                const float f = x.y != 0.f ? ex2_approx(least - x.x) : 0.f;
                sh.factor[w][tid] = f;
                if (x.y != 0.f) sum = fmaf(x.y, f, sum);
            }
            sh.joint[tid] = make_float2(least, sum);
        }
        consumer_sync();
        const float low = kLow / v_unit, high = kHigh / v_unit;
        constexpr int kQuads = (Q * 32 + kWarps * 32 - 1) / (kWarps * 32);
        float4 all[kQuads] = {};  // four channels of a query
#pragma unroll 1
        for (int first = 0; first < kWarps; first += 2) {
            if (warp >= first && warp < first + 2) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int col = nt * 8 + 2 * t + c;
                        const float f = sh.factor[warp][col];
                        float* dst = reinterpret_cast<float*>(sh.sums[warp - first][col]) + g;
                        const bool some = l[nt][c] != 0.f;
#pragma unroll
                        for (int cb = 0; cb < 8; ++cb) {
                            const float m = moff[nt][c][cb >> 2];
                            const float x = fmaf(out[nt][cb][c], low, m) * f;
                            const float y = fmaf(out[nt][cb][2 + c], high, m) * f;
                            dst[16 * cb] = some ? x : 0.f;
                            dst[16 * cb + 8] = some ? y : 0.f;
                        }
                    }
            }
            consumer_sync();
#pragma unroll
            for (int i = 0; i < kQuads; ++i) {
                const int quad = tid + i * kWarps * 32;
                if (quad >= Q * 32) break;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const float4 x = sh.sums[w][quad >> 5][quad & 31];
                    all[i].x += x.x;
                    all[i].y += x.y;
                    all[i].z += x.z;
                    all[i].w += x.w;
                }
            }
            consumer_sync();
        }
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const int quad = tid + i * kWarps * 32;
            if (quad >= Q * 32) break;
            const int c = quad >> 5, row = st.block * Q + c;
            const float2 joint = sh.joint[c];
            const float4 x = all[i];
            if (st.part >= 0) {
                const long long at = (long long)st.part * Q + c;
                reinterpret_cast<float4*>(a.part)[at * 32 + lane] = x;
                if (lane == 0)
                    reinterpret_cast<float2*>(a.part + 2LL * a.pieces * Q * D)[at] = joint;
            } else if (row < a.rows) {
                const float inv = joint.y == 0.f ? 0.f : 1.f / joint.y;
                const int i_row = row / a.group;
                const long long at = ((long long)st.n * a.krows + i_row) * a.heads +
                                     st.head * a.group + row - i_row * a.group;
                reinterpret_cast<uint2*>(a.o + at * D)[lane] = make_uint2(
                    narrow2<F16>(x.x * inv, x.y * inv), narrow2<F16>(x.z * inv, x.w * inv));
                if (a.lse && lane == 0)
                    a.lse[at] = joint.y == 0.f ? -INFINITY : (log2f(joint.y) - joint.x) * kLn2;
            }
        }
    }
}

template <bool F16, int NT>
__global__ void __launch_bounds__(kThreads, kCtas<NT>) attn_decode_kernel(DecodeArgs a) {
    extern __shared__ __align__(128) uint8_t sm[];
    Shared<NT>& sh = *reinterpret_cast<Shared<NT>*>(sm + kStages<NT> * kStageBytes);
    if (threadIdx.x == 0) {
        sh.stop = 0;
        for (int i = 0; i < kStages<NT>; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_release();
    if (threadIdx.x < kWarps * 32) attend_role<F16, NT>(a, sh, sm);
    else copy_role<NT>(a, sh, sm);
}

// Joins what several CTAs have of one (sequence, head, block), and writes rows
// that no CTA has anything of.  A warp takes some of the unit's query columns,
// four channels a lane.
constexpr int kJoinWarps = 16;
template <bool F16, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join_kernel(DecodeArgs a) {
    constexpr int Q = 8 * NT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_seq = a.c.kv_heads * a.blocks;
    const int n = blockIdx.x / per_seq, unit = blockIdx.x - n * per_seq;
    const int head = unit / a.blocks, block = unit - head * a.blocks;
    pdl_wait();
    long long before = 0;
    int count = 0;
    const long long one = scan_lengths(a, [&](int n0, long long b, int mine) {
        if (n >= n0 && n < n0 + 32) {
            before = __shfl_sync(0xffffffffu, b, n - n0);
            count = __shfl_sync(0xffffffffu, mine, n - n0);
        }
        return true;
    });
    const long long total = one * per_seq;
    int b0 = 0, b1 = -1, slot0 = 0;
    if (count) {
        const long long start = before * per_seq + (long long)unit * count;
        auto piece_of = [&](long long at) {
            const int pieces = piece_count(a, total);
            int b = (int)(at * pieces / total);
            while (b + 1 < pieces && piece_start(a, total, b + 1) <= at) ++b;
            while (piece_start(a, total, b) > at) --b;
            return b;
        };
        b0 = piece_of(start);
        b1 = piece_of(start + count - 1);
        if (b0 == b1) return;  // one CTA had all of it
        slot0 = 2 * b0 + (piece_start(a, total, b0) == start ? 0 : 1);
    }
    const float2* stat = reinterpret_cast<const float2*>(a.part + 2LL * a.pieces * Q * D);
    for (int c = warp; c < Q; c += kJoinWarps) {
        const int row = block * Q + c;
        if (row >= a.rows) break;
        float least = INFINITY;
        for (int b = b0 + lane; b <= b1; b += 32) {
            const float2 s = __ldcg(stat + (b == b0 ? slot0 : 2 * b) * Q + c);
            if (s.y != 0.f) least = fminf(least, s.x);
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1)
            least = fminf(least, __shfl_xor_sync(0xffffffffu, least, off));
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int from = b0; from <= b1; from += 32) {
            // a piece's factor and part of the sum a lane, then its 128 channels
            const int b = from + lane;
            float f = 0.f;
            if (b <= b1) {
                const float2 s = __ldcg(stat + (b == b0 ? slot0 : 2 * b) * Q + c);
                if (s.y != 0.f) {
                    f = ex2_approx(least - s.x);
                    sum = fmaf(s.y, f, sum);
                }
            }
            const int n_here = min(32, b1 - from + 1);
#pragma unroll 8
            for (int i = 0; i < n_here; ++i) {
                const int slot = from + i == b0 ? slot0 : 2 * (from + i);
                const float4 x = __ldcg(reinterpret_cast<const float4*>(
                                            a.part + ((long long)slot * Q + c) * D) + lane);
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
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const long long at = ((long long)n * a.krows + row / a.group) * a.heads + head * a.group +
                             row % a.group;
        *reinterpret_cast<uint2*>(a.o + at * D + 4 * lane) =
            make_uint2(narrow2<F16>(o.x * inv, o.y * inv), narrow2<F16>(o.z * inv, o.w * inv));
        if (a.lse && lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : (log2f(sum) - least) * kLn2;
    }
}

// Query columns of a block: 8 where that is all, else 16.
inline int columns(int rows) { return rows <= 8 ? 8 : 16; }

template <bool F16, int NT>
cudaError_t launch(const DecodeArgs& a, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<F16, NT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes<NT>());
    if (e != cudaSuccess) return e;
    launch_pdl(attn_decode_kernel<F16, NT>, dim3(a.pieces), dim3(kThreads), smem_bytes<NT>(), s, a);
    return launch_pdl(attn_join_kernel<F16, NT>,
                      dim3((unsigned)((long long)a.n_seqs * a.c.kv_heads * a.blocks)),
                      dim3(kJoinWarps * 32), 0, s, a);
}

}  // namespace

cudaError_t read_and_clear_status_decode(unsigned* out) {
    const unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_decode_status, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_decode_status, &zero, sizeof(unsigned));
    return e;
}

}  // namespace kda

using namespace kda;

// Two incomplete segments per CTA, 152 SMs' worth of CTAs (more on a device with
// more: see the call).
extern "C" size_t kda_attn_kv4_workspace_size(int n_seqs, int krows, int heads, int kv_heads) {
    if (n_seqs < 1 || krows < 1 || krows > KDA_MAX_K || heads < 1 || kv_heads < 1 ||
        heads % kv_heads)
        return 0;
    const size_t q = (size_t)columns(krows * (heads / kv_heads));
    return KDA_KV4_PIECES * 2 * q * (D + 2) * sizeof(float);
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
    const int ctas = (cols == 8 ? kCtas<1> : kCtas<2>) * sm_count();
    const int pieces = ctas < KDA_KV4_PIECES ? ctas : KDA_KV4_PIECES;
    KDA_REQUIRE(pieces > 0, KDA_ERR_CUDA, "%s: no device", fn);
    DecodeArgs a = {(const uint16_t*)q, (uint16_t*)o, lse, n_seqs, krows, heads, window, group,
                    rows, blocks, scale, pieces, static_cast<float*>(workspace),
                    {const_cast<uint8_t*>(cache), page_table, lens, n_pages, max_pages,
                     __builtin_ctz((unsigned)page), kv_heads}};
    cudaStream_t s = as_stream(stream);
    const bool f16 = in_dtype == KDA_F16;
    cudaError_t e;
    if (cols == 8) e = f16 ? launch<true, 1>(a, s) : launch<false, 1>(a, s);
    else e = f16 ? launch<true, 2>(a, s) : launch<false, 2>(a, s);
    if (e != cudaSuccess) {
        set_error("%s: launch failed: %s", fn, cudaGetErrorString(e));
        return KDA_ERR_CUDA;
    }
    return launch_result(fn);
}
