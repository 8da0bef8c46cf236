// Attention of 1..8 query rows per sequence over the paged 4-bit cache
// (kda_attn_kv4_decode): kda_attn_prefill's formula with the cache's values
// m + s * code as keys and values.
//
// HBM-bound: 144 bytes per (position, KV head), read once for all of the
// group's query heads and rows.  What the values cost on the way:
//  - Codes go to the matrix instructions as they are: with x = s (code - 8) +
//    (m + 8 s) and 64 channels to a step s,
//        q . k = sum_a s_a (q . (code - 8))_a + (m_a + 8 s_a) (sum q)_a
//        o_d   = sum_t (p_t s_ta) (code - 8)_td + sum_t p_t (m_ta + 8 s_ta)
//    so a code becomes a 16-bit number in about one operation and steps and
//    minima meet scores and weights, not values.
//  - The cache keeps codes in the order of mma.sync's A operand: keys (or value
//    channels) are the product's 16 rows, queries its 8 columns, so that one
//    query row in use wastes 7 of 8 columns of an instruction that is not the
//    bound, and no shared-memory transposition is needed.
//  - A score's columns are queries, as an output's are: running sums and
//    rescaling stay within a lane.  p_t s_ta is rounded to BF16 (8 significant
//    bits, FP32's range whatever s is); scores, sums and outputs are FP32.
//
// All positions of the batch, in chunks of 128 tokens, are one line that the
// CTAs cut into equal pieces, whatever the lengths: a piece ends where it ends,
// and what is left of a (sequence, head) in each is joined by a second kernel
// (attn_join_kernel), always in the same order.  Per CTA one warp copies chunks
// into a ring in shared memory, eight warps take 16 tokens of each.
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

constexpr int kChunk = 128;  // tokens
constexpr int kWarps = 8;    // of 16 tokens of each chunk
constexpr int kThreads = (kWarps + 1) * 32;
// With 16 query columns a thread needs more registers than two CTAs to a
// multiprocessor leave it.
template <int NT>
constexpr int kCtas = NT == 1 ? 2 : 1;
template <int NT>
constexpr int kStages = NT == 1 ? 4 : 8;
constexpr int kStageBytes = kChunk * kTokenBytes;  // K codes, V codes, K and V parameters
constexpr int kVCodes = kChunk * 64, kKPar = 2 * kVCodes, kVPar = kKPar + kChunk * 8;

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
    const int lo = a.window ? max(0, len - a.krows - a.window + 1) : 0;
    return {lo / kChunk, len > 0 ? (len - 1) / kChunk + 1 - lo / kChunk : 0};
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

// What a stage of the ring holds.
struct Stage {
    int n, head, block;  // block: of 8 NT query rows
    int pos;             // the chunk's first position
    uint32_t there;      // bit i: tokens 16 i .. 16 i + 15 are in the stage
    int start, end;      // of a segment: what one CTA does of one (n, head, block)
    int part;            // where an incomplete segment's sums go, or -1; -2: no more
};

template <int NT>
struct Shared {
    uint64_t full[kStages<NT>], empty[kStages<NT>];
    Stage stage[kStages<NT>];
    float2 stat[kWarps][8 * NT];  // a warp's (shift, l) by query
    float sums[4][128][8 * NT];   // half of the warps' outputs at a time
    int stop;
};
template <int NT>
constexpr int smem_bytes() {
    return kStages<NT> * kStageBytes + (int)sizeof(Shared<NT>);
}

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
    const int piece = min(a.c.page(), kChunk);       // tokens that lie together
    const int per_chunk = kChunk / piece;            // such pieces of a chunk
    const uint32_t groups = (1u << (piece / 16)) - 1;  // bits of `there`, one piece's
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
                const int first_page = pos >> a.c.page_shift;
                if (ids_from < 0 || first_page + per_chunk > ids_from + 32) {
                    ids_from = first_page;
                    const int p = first_page + lane;
                    ids = p < a.c.max_pages && ((long long)p << a.c.page_shift) < len
                              ? __ldg(table + p)
                              : -1;
                }
                const int id = __shfl_sync(0xffffffffu, ids, first_page - ids_from + lane);
                const bool wanted = lane < per_chunk && pos + lane * piece < len;
                const bool valid = wanted && id >= 0 && id < a.c.n_pages;
                if (wanted && !valid) atomicOr(&g_decode_status, STATUS_BAD_PAGES);
                const unsigned ok = __ballot_sync(0xffffffffu, valid);
                uint32_t there = 0;
                for (int i = 0; i < per_chunk; ++i)
                    if (ok >> i & 1) there |= groups << (i * (piece / 16));
                go = wait_warp(sh, &sh.empty[stage], phase ^ 1);
                if (!go) break;
                if (lane == 0) {
                    sh.stage[stage] = {n, head, block, pos, there, at == seg_start,
                                       at + 1 == seg_end, part};
                    mbar_arrive_expect_tx(&sh.full[stage],
                                          (uint32_t)__popc(ok) * piece * kTokenBytes);
                }
                __syncwarp();
                if (valid) {
                    const int in_page = (pos & (a.c.page() - 1));
                    const uint8_t* src = a.c.data +
                                         ((long long)id * heads + head) * a.c.block_bytes();
                    uint8_t* dst = sm + stage * kStageBytes;
                    const int tok = lane * piece;
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const uint8_t* part_src = src + v * part_bytes(a.c.page());
                        bulk_load(dst + v * kVCodes + tok * 64, part_src + in_page * 64,
                                  piece * 64, &sh.full[stage]);
                        bulk_load(dst + kKPar + v * kChunk * 8 + tok * 8,
                                  part_src + a.c.page() * 64 + in_page * 8, piece * 8,
                                  &sh.full[stage]);
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
            sh.stage[stage].part = -2;
            mbar_arrive(&sh.full[stage]);
        } else {
            // copies in flight land before the CTA's memory goes away
            for (int s = 0; s < kStages<NT>; ++s)
                mbar_wait(&sh.full[s], s < stage ? phase : phase ^ 1, 1 << 12);
        }
    }
}

__device__ __forceinline__ uint32_t sub_h2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t sub_b2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// A word of codes as the A operand: codes - 8 in FP16.  The low four bits of a
// byte make 1024 + code in place, the high four 64 + code.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&a)[4]) {
    const uint32_t v = w >> 8;
    a[0] = sub_h2((w & 0x000f000fu) | 0x64006400u, 0x64086408u);
    a[2] = sub_h2((w & 0x00f000f0u) | 0x54005400u, 0x54805480u);
    a[1] = sub_h2((v & 0x000f000fu) | 0x64006400u, 0x64086408u);
    a[3] = sub_h2((v & 0x00f000f0u) | 0x54005400u, 0x54805480u);
}
// The same in BF16, where 128 + code is made; rows g + 8 are the high four bits.
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t (&a)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = sub_b2((w >> (4 * i) & 0x000f000fu) | 0x43004300u, 0x43084308u);
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
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

// 2^x for x <= 0, 0 for -inf.
__device__ __forceinline__ float pow2(float x) { return ex2_approx(x); }

template <bool F16, int NT>
__device__ __forceinline__ void attend_role(const DecodeArgs& a, Shared<NT>& sh,
                                            const uint8_t* sm) {
    constexpr int Q = 8 * NT;  // query columns
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    int stage = 0;
    uint32_t phase = 0;
    // the segment's queries: B operands (FP16, scaled by a power of two), the
    // factor from a product to a score in log2 units and the sums over 64
    // channels, of columns 8 nt + 2 t + e
    uint32_t qb[NT][8][2];
    float unit[NT][2], qsum[NT][2][2];
    int limit[NT][2], lo[NT][2];  // positions a column sees: [lo, limit)
    int clear_lo = 0, clear_hi = 0;
    float out[NT][8][4];
    float shift[NT][2], l[NT][2], moff[NT][2][2];  // moff: sum p (m + 8 s), by 64 channels
    bool settled = false;  // every column has a shift that comes from a score
    for (;;) {
        if (!wait_warp(sh, &sh.full[stage], phase)) return;
        const Stage st = sh.stage[stage];
        if (st.part == -2) return;
        if (st.start) {
            const int len = good_len(a, __ldg(a.c.lens + st.n));
            clear_hi = len - a.krows + 1;
            clear_lo = a.window ? max(0, len - a.window) : 0;
            settled = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // the row of B column g
                const int row = st.block * Q + nt * 8 + g;
                const int i = row / a.group, hh = row - i * a.group;
                const bool there = row < a.rows;
                const uint32_t* src = reinterpret_cast<const uint32_t*>(
                    a.q + (((long long)st.n * a.krows + (there ? i : 0)) * a.heads +
                           st.head * a.group + (there ? hh : 0)) * D);
                uint32_t raw[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) raw[k] = there ? __ldg(src + 4 * k + t) : 0u;
                float big = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float2 x = widen2<F16>(raw[k]);
                    big = fmaxf(big, fmaxf(fabsf(x.x), fabsf(x.y)));
                }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                // bring the largest to 2^14..2^15: exact, and what is below FP16's
                // smallest number then is 2^-38 of it
                const int e = (int)(__float_as_uint(big) >> 23) - 127;
                const bool plain = big == 0.f || !(big < INFINITY);
                const int up = plain ? 0 : max(-126, min(126, 14 - e));
                const float f = __uint_as_float((uint32_t)(127 + up) << 23);
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float2 x = widen2<F16>(raw[k]);
                    x.x *= f;
                    x.y *= f;
                    if (k < 8) s0 += x.x + x.y;
                    else s1 += x.x + x.y;
                    qb[nt][k >> 1][k & 1] = narrow2<true>(x.x, x.y);
                }
                s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
                s0 += __shfl_xor_sync(0xffffffffu, s0, 2);
                s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
                s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
                const float un =
                    a.scale * kLog2e * __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = 2 * t + c;  // its values are with lanes 4 col ..
                    unit[nt][c] = __shfl_sync(0xffffffffu, un, 4 * col);
                    qsum[nt][c][0] = __shfl_sync(0xffffffffu, s0, 4 * col);
                    qsum[nt][c][1] = __shfl_sync(0xffffffffu, s1, 4 * col);
                    const int crow = st.block * Q + nt * 8 + col;
                    const int ci = crow / a.group;
                    limit[nt][c] = crow < a.rows ? len - a.krows + ci + 1 : 0;
                    lo[nt][c] = a.window ? max(0, limit[nt][c] - a.window) : 0;
                    shift[nt][c] = l[nt][c] = 0.f;
                    moff[nt][c][0] = moff[nt][c][1] = 0.f;
                }
#pragma unroll
                for (int cb = 0; cb < 8; ++cb)
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) out[nt][cb][i4] = 0.f;
            }
        }
        const int pos = st.pos + 16 * warp;
        if (st.there >> warp & 1) {
            const uint8_t* base = sm + stage * kStageBytes;
            // scores of tokens g and g + 8
            uint32_t kw[8];
            {
                const uint4* p = reinterpret_cast<const uint4*>(base + warp * 1024) + lane;
                const uint4 x = p[0], y = p[32];
                kw[0] = x.x, kw[1] = x.y, kw[2] = x.z, kw[3] = x.w;
                kw[4] = y.x, kw[5] = y.y, kw[6] = y.z, kw[7] = y.w;
            }
            const uint2* kp = reinterpret_cast<const uint2*>(base + kKPar) + warp * 16 + g;
            const uint2 kpar[2] = {kp[0], kp[8]};
            float y[NT][4];
            {
                float acc[NT][2][4] = {};
#pragma unroll
                for (int kb = 0; kb < 8; ++kb) {
                    uint32_t ca[4];
                    codes_f16(kw[kb], ca);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(acc[nt][kb >> 2], ca, qb[nt][kb][0], qb[nt][kb][1]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float sa = __uint_as_float(kpar[i].x << 16);
                    const float ma = fmaf(8.f, sa, __uint_as_float(kpar[i].x & 0xffff0000u));
                    const float sb = __uint_as_float(kpar[i].y << 16);
                    const float mb = fmaf(8.f, sb, __uint_as_float(kpar[i].y & 0xffff0000u));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float d = ma * qsum[nt][c][0];
                            d = fmaf(mb, qsum[nt][c][1], d);
                            d = fmaf(sa, acc[nt][0][2 * i + c], d);
                            d = fmaf(sb, acc[nt][1][2 * i + c], d);
                            y[nt][2 * i + c] = d * unit[nt][c];
                        }
                }
            }
            const bool edge = pos < clear_lo || pos + 16 > clear_hi;
            if (edge) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = pos + g + 8 * (i >> 1);
                        if (at < lo[nt][i & 1] || at >= limit[nt][i & 1]) y[nt][i] = -INFINITY;
                    }
            }
            // shifts: from the first scores of a column, and again once a weight
            // would pass 2^30
            bool over = !settled;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    over |= fmaxf(y[nt][c], y[nt][2 + c]) + shift[nt][c] > 30.f;
            if (__any_sync(0xffffffffu, over)) {
                bool all = true;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float top = max_keys(fmaxf(y[nt][c], y[nt][2 + c]));
                        const bool fresh = sum_keys(l[nt][c]) == 0.f;
                        const bool move = top > -INFINITY && (fresh || top + shift[nt][c] > 30.f);
                        const float f = fresh || !move ? 1.f : pow2(-top - shift[nt][c]);
                        if (move) shift[nt][c] = -top;
                        l[nt][c] *= f;
                        moff[nt][c][0] *= f;
                        moff[nt][c][1] *= f;
#pragma unroll
                        for (int cb = 0; cb < 8; ++cb) {
                            out[nt][cb][c] *= f;
                            out[nt][cb][2 + c] *= f;
                        }
                        // a column that will see a key later has no shift yet
                        all &= !fresh || move || limit[nt][c] <= pos + 16;
                    }
                settled = __all_sync(0xffffffffu, all);
            }
            // weights, and with the values' steps the second product's B operand
            const uint2* vp = reinterpret_cast<const uint2*>(base + kVPar) + warp * 16 + g;
            const uint2 vpar[2] = {vp[0], vp[8]};
            uint32_t pb[NT][2][2];  // [64 channels][tokens 0..7, 8..15]
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float s[2], m[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w = h ? vpar[i].y : vpar[i].x;
                    s[h] = __uint_as_float(w << 16);
                    m[h] = fmaf(8.f, s[h], __uint_as_float(w & 0xffff0000u));
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float p0 = ex2_approx(y[nt][2 * i] + shift[nt][0]);
                    const float p1 = ex2_approx(y[nt][2 * i + 1] + shift[nt][1]);
                    l[nt][0] += p0;
                    l[nt][1] += p1;
                    // what a column does not see has no influence on it, a step
                    // or minimum that is NaN included
                    const bool no0 = edge && y[nt][2 * i] == -INFINITY;
                    const bool no1 = edge && y[nt][2 * i + 1] == -INFINITY;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!no0) moff[nt][0][h] = fmaf(p0, m[h], moff[nt][0][h]);
                        if (!no1) moff[nt][1][h] = fmaf(p1, m[h], moff[nt][1][h]);
                        pb[nt][h][i] = transpose8(
                            narrow2<false>(no0 ? 0.f : p0 * s[h], no1 ? 0.f : p1 * s[h]));
                    }
                }
            }
            uint32_t vw[8];
            {
                const uint4* p =
                    reinterpret_cast<const uint4*>(base + kVCodes + warp * 1024) + lane;
                const uint4 x = p[0], z = p[32];
                vw[0] = x.x, vw[1] = x.y, vw[2] = x.z, vw[3] = x.w;
                vw[4] = z.x, vw[5] = z.y, vw[6] = z.z, vw[7] = z.w;
            }
#pragma unroll
            for (int cb = 0; cb < 8; ++cb) {
                uint32_t ca[4];
                codes_bf16(vw[cb], ca);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_bf16(out[nt][cb], ca, pb[nt][cb >> 2][0], pb[nt][cb >> 2][1]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[stage]);
        if (++stage == kStages<NT>) stage = 0, phase ^= 1;
        if (!st.end) continue;

        // the segment's end: eight warps' sums become one
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                l[nt][c] = sum_keys(l[nt][c]);
                const float m0 = sum_keys(moff[nt][c][0]), m1 = sum_keys(moff[nt][c][1]);
#pragma unroll
                for (int cb = 0; cb < 8; ++cb) {
                    out[nt][cb][c] += cb < 4 ? m0 : m1;
                    out[nt][cb][2 + c] += cb < 4 ? m0 : m1;
                }
                if (g == 0) sh.stat[warp][nt * 8 + 2 * t + c] = make_float2(shift[nt][c], l[nt][c]);
            }
        consumer_sync();
        float total[NT][2], common[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                // the least shift is that of the largest score
                float least = INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 s = sh.stat[w][nt * 8 + 2 * t + c];
                    if (s.y != 0.f) least = fminf(least, s.x);
                }
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 s = sh.stat[w][nt * 8 + 2 * t + c];
                    if (s.y != 0.f) sum = fmaf(s.y, pow2(least - s.x), sum);
                }
                const float f = l[nt][c] != 0.f ? pow2(least - shift[nt][c]) : 0.f;
#pragma unroll
                for (int cb = 0; cb < 8; ++cb) {
                    out[nt][cb][c] = l[nt][c] != 0.f ? out[nt][cb][c] * f : 0.f;
                    out[nt][cb][2 + c] = l[nt][c] != 0.f ? out[nt][cb][2 + c] * f : 0.f;
                }
                total[nt][c] = sum;
                common[nt][c] = least;
            }
        for (int half = kWarps / 2; half >= 1; half /= 2) {
            if (warp >= half && warp < 2 * half) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int cb = 0; cb < 8; ++cb)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            *reinterpret_cast<float2*>(
                                &sh.sums[warp - half][16 * cb + g + 8 * i][8 * nt + 2 * t]) =
                                make_float2(out[nt][cb][2 * i], out[nt][cb][2 * i + 1]);
            }
            consumer_sync();
            if (warp < half) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int cb = 0; cb < 8; ++cb)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 x = *reinterpret_cast<const float2*>(
                                &sh.sums[warp][16 * cb + g + 8 * i][8 * nt + 2 * t]);
                            out[nt][cb][2 * i] += x.x;
                            out[nt][cb][2 * i + 1] += x.y;
                        }
            }
        }
        if (warp == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (g == 0)
                        sh.stat[0][nt * 8 + 2 * t + c] = make_float2(common[nt][c], total[nt][c]);
                }
#pragma unroll
                for (int cb = 0; cb < 8; ++cb)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        *reinterpret_cast<float2*>(&sh.sums[0][16 * cb + g + 8 * i][8 * nt + 2 * t]) =
                            make_float2(out[nt][cb][2 * i], out[nt][cb][2 * i + 1]);
            }
        }
        consumer_sync();
        const int tid = threadIdx.x;
        if (st.part >= 0) {
            float* dst = a.part + (long long)st.part * Q * D;
            for (int i = tid; i < Q * D; i += kWarps * 32) dst[i] = sh.sums[0][i & (D - 1)][i / D];
            float2* stat = reinterpret_cast<float2*>(a.part + 2LL * a.pieces * Q * D);
            if (tid < Q) stat[st.part * Q + tid] = sh.stat[0][tid];
        } else {
            for (int i = tid; i < Q * D / 2; i += kWarps * 32) {
                const int c = i / (D / 2), d = 2 * (i & (D / 2 - 1));
                const int row = st.block * Q + c;
                if (row >= a.rows) continue;
                const float sum = sh.stat[0][c].y;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const long long at = ((long long)st.n * a.krows + row / a.group) * a.heads +
                                     st.head * a.group + row % a.group;
                *reinterpret_cast<uint32_t*>(a.o + at * D + d) =
                    narrow2<F16>(sh.sums[0][d][c] * inv, sh.sums[0][d + 1][c] * inv);
                if (a.lse && d == 0)
                    a.lse[at] = sum == 0.f ? -INFINITY : (log2f(sum) - sh.stat[0][c].x) * kLn2;
            }
        }
        consumer_sync();  // the next segment's sums go to the same place
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
constexpr int kJoinWarps = 8;
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
#pragma unroll 8
        for (int b = b0; b <= b1; ++b) {
            const int slot = b == b0 ? slot0 : 2 * b;
            const float2 s = __ldcg(stat + slot * Q + c);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(
                                        a.part + ((long long)slot * Q + c) * D) + lane);
            if (s.y == 0.f) continue;
            const float f = pow2(least - s.x);
            sum = fmaf(s.y, f, sum);
            o.x = fmaf(x.x, f, o.x);
            o.y = fmaf(x.y, f, o.y);
            o.z = fmaf(x.z, f, o.z);
            o.w = fmaf(x.w, f, o.w);
        }
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
