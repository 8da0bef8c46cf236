// Linear attention with a decay for each head over prompts (kda_lin_prefill), in
// chunks of C = 128 tokens on the tensor cores.  With G_t the sum of g over a chunk's
// tokens up to t, S the state in front of the chunk and a head's Q, K, V [C][128],
//     P[t][s] = exp(G_t - G_s) (Q K^T)[t][s] for s <= t, else 0
//     O = scale * (P V + diag(exp(G_t)) Q S)
//     S <- exp(G_C) S + K^T W,      W[s] = exp(G_C - G_s) V[s]
//
// Bound by memory: 1 KB a token and head, 0.15 ns, for five 128^3 products a chunk and head,
// 164 kFLOP a token and head, 0.09 ns.  So all of a chunk's work has to fit under its copy,
// 2.9 us at a multiprocessor's share of the bandwidth:
//  - One persistent CTA a multiprocessor, chunks one after the other; chunk c + 1's
//    Q, K and V are copied by TMA while chunk c is worked on.
//  - S stays in registers, FP32, added to with one rounding a chunk (256 threads, a row
//    of 64 columns each); the products' accumulators are TMEM's four quarters: Q K^T (P
//    is written over it), Q S, P V, K^T W.
//  - Decays never enter as exp(G_t) exp(-G_s), whose factors leave FP32's range.  Below
//    the diagonal blocks of 32 tokens the factors are decays up to the end of s's block
//    and from there to t, on them exp(G_t - G_s) itself.  Sums of g run within blocks, and
//    those of blocks with very strong decays in two parts (deep_decays), so that decays near 1
//    do not come from differences of large sums.
//  - P and the copy of S that Q is multiplied with are rounded to 16 bits, as tensor cores
//    take them: O is off by half a 16-bit step of the sums of |P V| and |Q S|, about as much
//    again as by its own rounding (more where terms cancel).  W is kept as two 16-bit
//    numbers, hi + lo, and the product done twice: the state accumulates over thousands of
//    tokens and is an FP32 output.  hi is written over V and lo over Q once both are
//    through, so that two stages of inputs fit.
//  - FP16 operands are scaled by powers of two that the largest entry of S, or of V,
//    in the chunk gives, weights by one that their row's largest product gives: FP16's range
//    is narrower than FP32 states and products are.
//
// Pieces.  All chains (heads of sequences), one after the other, are cut into equal pieces,
// one a CTA.  Where no chain is longer than a piece, a CTA works on the beginning of its last
// chain first of all and hands the state on, and on the end of its first one last.  (For chains
// up to half as long again pieces are made as long as they are, and some CTAs have none.)
// Longer chains, which lie in several pieces, need the state in front of them early:
// lin_prefill_kernel<.., SUM> first adds up what each cut segment contributes (K and V
// alone).  See Plan.
//
// A chunk takes 3.3 to 3.4 us, a CTA's first 7 us more and a change of chains 5: 16 prompts of
// 512 to 8192 tokens, 32 heads (2.4 GB): 449 us, 5.3 TB/s.  One prompt of 8192 tokens, 32
// heads (0.27 GB): 101 us, of these 38 for the sums; FP16: 123.
#include <algorithm>
#include <cmath>
#include <cstddef>

#include "f32x2.h"
#include "lin_attn.h"
#include "sm103_tc.h"
#include "tma_map.h"

namespace kda {
namespace {

using namespace attn;
using namespace tc;
using lin::Args;

__device__ unsigned g_lin_status = 0;

constexpr int C = 128;  // tokens a chunk
constexpr int kSms = 152;
// A piece's chunks at least (4: 1500 tokens, 32 heads 38 us, 3: 33; 2: some calls are better
// off by a sixth, others worse).
constexpr int kLeastPiece = 3;
// Calls of so few chunks, and of a chain a CTA at most, cut none: one kernel (700 tokens, 24
// heads: 25.7 us, with cuts 30.2).
constexpr int kWhole = 6;
constexpr int kStateFloats = D * D;

// ---------------------------------------------------------------- pieces

// How the call's chunks go to `pieces` CTAs (at most kSms).
//  kPadded: each chain starts a piece, pieces of kLeastPiece (kWhole) chunks: few chunks.
//  kEven: chains one after the other, cut into equal pieces.  A chain counts kLead chunks
//      more than it has, in front of its first one: what its states' load and store cost.
//      (kLead 1: 16 prompts of 512 to 8192 tokens in this order, 32 heads, 462 us, 2: 422.)
//  kHandOver: the same where no chain is longer than a piece, so that none lies in more
//      than two, or where pieces as long as the longest chain cost less than sums do.
//      (Whole chains dealt out by length: the same at many chains, but 114 us for 5 prompts
//      of 2048 tokens, 32 heads, where this takes 87.)
enum Kind { kPadded, kEven, kHandOver };
constexpr int kLead = 2;
// By the model 3.4 us a chunk and 12 in all, the sums 2 us a chunk and 12: 4 prompts of 2048
// tokens, 32 heads, 78 us; cut into 152 pieces, with sums, 103.  (2 prompts: 74, and 67.)
__host__ __device__ __forceinline__ bool hand_over(long long longest, long long piece) {
    return longest + kLead <= piece + piece / 2 + 3;
}
// Part of one chain: chunks [from, to) of the `of` that head h of sequence n has.
struct Segment {
    int n, h, from, to, of;
};
struct Plan {
    Kind kind;
    int piece;        // units of a piece: chunks, with chains' lead
    long long total;  // units, or (kPadded) pieces

    // Pieces of a segment's chain in front of its last one, at most.
    __device__ __forceinline__ int chain_folds(const Segment& s) const { return s.of / piece + 1; }
    // The piece in which a chain begins, of whose chunks piece i starts with number `from`.
    __device__ __forceinline__ int chain_begin(int i, int from) const {
        return kind == kPadded ? i - from / piece
                               : (int)(((long long)i * piece - from) / piece);
    }
};
struct Work {
    Args a;
    int pieces;
    int least;  // chunks of a piece: kLeastPiece, or kWhole if no chain is longer
    // of a piece whose last segment's chain goes on in the next piece: what the segment
    // adds to the state, then the state in front of the next piece
    float* sum;      // [pieces][128 * 128]
    float* log_sum;  // [pieces] log2 of the segment's decay
    float* start;    // [pieces] the state in front of a cut chain that starts there, where
                     // state_out is state_in
    float* folded;   // [pieces] the state in front of a piece
    unsigned* handed;  // [pieces] kHandOver: 1 once `sum` is the state of its last chain
};
// A segment's state is summed up where it is wanted from at most so many pieces before it
// (a microsecond each, what 64 KB from L2 take); of longer chains by lin_join_kernel (7 us: one
// chain in 17 pieces 37.9 us, folded 40.7).
constexpr int kMostFolds = 14;

__device__ __forceinline__ int chunks_of(const Args& a, int n) {
    lin::Rows r;
    return sequence_rows(a, n, r) ? (r.count + C - 1) / C : 0;
}
__device__ __forceinline__ int padded(int chunks, int least) {
    return (chunks + least - 1) / least;
}

__device__ __forceinline__ int units(int chunks) { return chunks ? chunks + kLead : 0; }
// The chunk in front of which unit u of a chain begins.
__device__ __forceinline__ int chunk_at(int u) { return max(0, u - kLead); }

// One warp; the same for all warps of the call.
__device__ __forceinline__ Plan make_plan(const Work& w) {
    const Args& a = w.a;
    const int lane = threadIdx.x & 31;
    long long chunks = 0, pads = 0;
    int longest = 0;
    if (!a.cu) {
        longest = (a.t + C - 1) / C;
        chunks = (long long)(longest + kLead) * a.n_seqs;
        pads = (long long)padded(longest, w.least) * a.n_seqs;
    } else {
        for (int n = lane; n < a.n_seqs; n += 32) {
            const int c = chunks_of(a, n);
            chunks += units(c);
            pads += padded(c, w.least);
            longest = max(longest, c);
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            chunks += __shfl_xor_sync(0xffffffffu, chunks, off);
            pads += __shfl_xor_sync(0xffffffffu, pads, off);
            longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, off));
        }
    }
    chunks *= a.heads;
    pads *= a.heads;
    const bool few = pads <= w.pieces;
    if (few && (longest <= w.least || !hand_over(longest, w.least)))
        return {kPadded, w.least, pads};
    const int piece =
        few ? w.least : (int)max((chunks + w.pieces - 1) / w.pieces, (long long)w.least);
    if (hand_over(longest, piece)) return {kHandOver, max(piece, units(longest)), chunks};
    return {kEven, piece, chunks};
}

// The chain that unit x falls in (kPadded: that piece x of `pads` chunks is of; otherwise
// `pads` is 0), x below the total;
// returns x's number within it.  One warp.
__device__ __forceinline__ int find_chain(const Args& a, int pads, long long x, int& n, int& h) {
    if (!a.cu) {
        const int c = (a.t + C - 1) / C, u = pads ? padded(c, pads) : units(c);
        const long long chain = x / u;
        n = (int)(chain / a.heads);
        h = (int)(chain - (long long)n * a.heads);
        return (int)(x - chain * u);
    }
    const int lane = threadIdx.x & 31;
    for (int n0 = 0; n0 < a.n_seqs; n0 += 32) {
        int u = 0;
        if (n0 + lane < a.n_seqs) {
            u = chunks_of(a, n0 + lane);
            u = pads ? padded(u, pads) : units(u);
        }
        long long sum = (long long)u * a.heads;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += up;
        }
        const long long all = __shfl_sync(0xffffffffu, sum, 31);
        if (x >= all) {
            x -= all;
            continue;
        }
        const unsigned past = __ballot_sync(0xffffffffu, sum > x);
        const int at = __ffs(past) - 1;
        const long long first = __shfl_sync(0xffffffffu, sum - (long long)u * a.heads, at);
        const int each = __shfl_sync(0xffffffffu, u, at);
        n = n0 + at;
        h = (int)((x - first) / each);
        return (int)(x - first - (long long)h * each);
    }
    n = h = 0;
    return 0;
}

// Goes through a piece's segments; the whole warp calls it.
struct Walk {
    Plan p;
    long long x, end;  // units still to come (kPadded: x is 0, then 1)
    int n, h, of, at;  // the chain that x falls in, its chunks, and x's number within it
    // kHandOver: the last segment, if its chain goes on in the next piece, comes first, and
    // the first one, if its chain began in the piece before, last.
    Segment head, tail;
    bool has_head = false, has_tail = false;

    __device__ __forceinline__ void begin(const Args& a, const Plan& plan, int piece) {
        p = plan;
        x = end = 0;
        if (p.kind == kPadded) return;
        x = (long long)piece * p.piece;
        end = min(p.total, x + p.piece);
        if (x >= end) return;
        at = find_chain(a, 0, x, n, h);
        of = chunks_of(a, n);
        if (p.kind == kEven) return;
        tail = {n, h, chunk_at(at), of, of};
        has_tail = tail.from > 0;
        if (has_tail) x += units(of) - at;
        if (x >= end) return;
        if (has_tail) next_chain(a);
        const int last = find_chain(a, 0, end - 1, head.n, head.h) + 1;
        head.from = 0;
        head.to = chunk_at(last);
        head.of = chunks_of(a, head.n);
        if (head.to < head.of) {  // (with no chunk of it here, it begins in the next piece)
            has_head = head.to > 0;
            end -= last;
        }
    }
    // (step by step, as finding a chain reads all offsets before it: 4096 prompts of 9 tokens, 2
    // heads, 2870 us, 603)
    __device__ __forceinline__ void next_chain(const Args& a) {
        at = 0;
        if (++h < a.heads) return;
        h = 0, ++n;
        if (!a.cu) return;
        const int lane = threadIdx.x & 31;
        for (; n < a.n_seqs; n += 32) {
            const int c = n + lane < a.n_seqs ? chunks_of(a, n + lane) : 0;
            const unsigned some = __ballot_sync(0xffffffffu, c > 0);
            if (!some) continue;
            of = __shfl_sync(0xffffffffu, c, __ffs(some) - 1);
            n += __ffs(some) - 1;
            return;
        }
    }
    __device__ __forceinline__ bool next(const Args& a, int piece, Segment& s) {
        if (p.kind == kPadded) {
            if (x++ || piece >= p.total) return false;
            const int part = find_chain(a, p.piece, piece, s.n, s.h);
            s.of = chunks_of(a, s.n);
            s.from = part * p.piece;
            s.to = min(s.of, s.from + p.piece);
            return true;
        }
        if (has_head) {
            has_head = false;
            s = head;
            return true;
        }
        while (x < end) {
            const int to = (int)min((long long)units(of), at + (end - x));
            s = {n, h, chunk_at(at), chunk_at(to), of};
            x += to - at;
            if (x < end) next_chain(a);
            if (s.from < s.to) return true;
        }
        if (!has_tail) return false;
        has_tail = false;
        s = tail;
        return true;
    }
};

// The last segment of piece i, if its chain goes on in the next one and its sum is wanted
// there.
__device__ __forceinline__ bool open_segment(const Work& w, const Plan& p, int i, Segment& s) {
    if (p.kind == kHandOver) return false;
    if (p.kind == kPadded) {
        if (i >= p.total) return false;
        const int part = find_chain(w.a, p.piece, i, s.n, s.h);
        s.of = chunks_of(w.a, s.n);
        s.from = part * p.piece;
        s.to = min(s.of, s.from + p.piece);
        return s.to < s.of;
    }
    const long long first = (long long)i * p.piece, end = min(p.total, first + p.piece);
    if (first >= end) return false;
    const int last = find_chain(w.a, 0, end - 1, s.n, s.h);
    s.of = chunks_of(w.a, s.n);
    s.to = chunk_at(last + 1);
    s.from = chunk_at((int)max(0LL, last - (end - 1 - first)));
    return s.from < s.to && s.to < s.of;
}

// ---------------------------------------------------------------- the kernel

// Warps: 0..3 P, 4..11 W, O and the state, 12 copies, 13 products, 14 and 15 look at
// V.
constexpr int kThreads = 512;
constexpr uint32_t kTile = C * D * 2;         // 32 KB
// Two stages of Q, K, V (later lo, K, hi) and S in 16 bits; SUM: three of K, V (K, hi) and lo.
constexpr uint32_t kStage = 3 * kTile, kSumStage = 2 * kTile;
constexpr uint32_t kStateTile = 2 * kStage;
static_assert(3 * kSumStage == kStateTile, "lo where S is otherwise");
template <bool SUM>
constexpr int kStages = SUM ? 3 : 2;
constexpr uint32_t kTmemP = 0, kTmemQS = 128, kTmemPV = 256, kTmemKW = 384;
constexpr int kRing = 2;

struct Item {
    int row, rows;  // the segment's first token row, and how many
    int h;
    int chunks;     // 0: no more segments
    const float* src;  // the state in front; null: zeros (SUM: a state to be copied)
    int fold, folds;   // pieces whose sums go on top: the first one, how many
    const unsigned* wait;  // kHandOver: src is there once this is 1; null: it is there
    unsigned* hand;        // dst is handed over by this; null: it is not
    float* dst;        // where the state behind goes; null: nowhere
};

struct Shared {
    uint64_t full[3], v_full[2], empty[3];
    uint64_t qk_ready, pv_ready, s16_ready, qs_ready;
    // by chunk parity, where one side may be a chunk ahead of the other's wait
    uint64_t p_ready[2], v_checked[2], w_ready[2], kw_ready[2], o_read[2];
    uint64_t token_sync, state_sync;
    uint64_t item_full[kRing], item_empty[kRing];
    Item item[kRing];
    uint32_t tmem;
    int stop;
    // within blocks of 32 tokens: less the sum of g (log2) up to each token, and the decay
    // behind it
    alignas(16) float sum[C];
    alignas(16) float tail[2][C];
    float front[C];        // scale * the decay from the chunk's start to each token
    uint8_t weight_unit[C];  // FP16: what each token's weights are in units of (exponent)
    float later[2][4];     // decay of the blocks behind each block
    float total[2];        // sum of the chunk
    float block[2][4];     // sums of blocks
    float largest[2][8];   // FP16: of S (SUM: of V), each warp's
    uint32_t most_v[2][2]; // FP16: the largest magnitude in each half of V
    // V's infinities and NaN, by chunk parity: each column's first token (255: none)
    uint32_t bad_first[2][D / 4];
    int bad[2], bad_seen[2];  // whether there are any; warps that are through with them
};
constexpr uint32_t kSharedOff = kStateTile + kTile;
constexpr uint32_t kSmemBytes = kSharedOff + sizeof(Shared);
static_assert(kSmemBytes <= 232448, "shared memory");
static_assert(offsetof(Shared, sum) % 16 == 0 && offsetof(Shared, tail) % 16 == 0 &&
                  kSharedOff % 16 == 0, "read by 16 bytes");

// Waits with an end: a phase that does not come within 2^35 clocks (some 17
// seconds), or another role's giving up, ends the kernel with an error status.
__device__ __noinline__ bool wait_long(Shared& sh, uint64_t* bar, uint32_t parity) {
    const long long from = clock64();
    while (!mbar_wait(bar, parity, 32)) {
        if (*(volatile int*)&sh.stop) return false;
        if (clock64() - from > 1LL << 35) {
            atomicOr(&g_lin_status, STATUS_TIMEOUT);
            *(volatile int*)&sh.stop = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_warp(Shared& sh, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, 1) || wait_long(sh, bar, parity));
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(yes));
    return yes != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
// A barrier among some warps, with an end like the other waits (bar.sync has none).
__device__ __forceinline__ bool sync_warps(Shared& sh, uint64_t* bar, uint32_t& phase) {
    arrive_warp(bar);
    const bool ok = wait_warp(sh, bar, phase);
    phase ^= 1;
    return ok;
}

// The roles' view of the ring of segments.  A segment is read where it lies, so that it
// takes no registers, and given back by `done`.
struct Items {
    int ring = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ const Item* next(Shared& sh) {  // null: no more
        if (!wait_warp(sh, &sh.item_full[ring], phase)) return nullptr;
        const Item* it = &sh.item[ring];
        if (it->chunks > 0) return it;
        done(sh);
        return nullptr;
    }
    __device__ __forceinline__ void done(Shared& sh) {
        arrive_warp(&sh.item_empty[ring]);
        if (++ring == kRing) ring = 0, phase ^= 1;
    }
};

// The copying warp: hands out segments and fills the stages.  (Tiles pulled into L2 one
// to three chunks ahead of that: no faster.)
template <bool SUM>
__device__ __forceinline__ void copy_role(const Work& w, Shared& sh, unsigned char* sm,
                                          const CUtensorMap* mq, const CUtensorMap* mk,
                                          const CUtensorMap* mv) {
    const Args& a = w.a;
    const int lane = threadIdx.x & 31, piece = blockIdx.x;
    const Plan plan = make_plan(w);
    Walk walk;
    walk.begin(a, plan, piece);
    Segment cut;
    bool done = SUM && !open_segment(w, plan, piece, cut), go = true;
    int ring = 0, stage = 0;
    uint32_t ring_phase = 0, phase = 0;
    while (go) {
        Item it = {};
        Segment s = cut;
        if (!done && (SUM || walk.next(a, piece, s))) {
            lin::Rows r;
            sequence_rows(a, s.n, r);
            it.row = (int)r.first + s.from * C;
            it.rows = min(r.count - s.from * C, (s.to - s.from) * C);
            it.h = s.h;
            it.chunks = s.to - s.from;
            const size_t chain = ((size_t)s.n * a.heads + s.h) * kStateFloats;
            if (SUM) {
                it.dst = w.sum + (size_t)piece * kStateFloats;
                // the state in front of a chain that is cut is kept where the chain's end
                // may be written before its beginning is read
                if (s.from == 0 && a.state_in && a.state_in == a.state_out)
                    it.src = a.state_in + chain;
                done = true;
            } else {
                if (plan.kind == kHandOver) {
                    it.src = a.state_in ? a.state_in + chain : nullptr;
                    if (s.from) {
                        it.src = w.sum + (size_t)(piece - 1) * kStateFloats;
                        it.wait = w.handed + piece - 1;
                    }
                    if (s.to < s.of) {
                        it.dst = w.sum + (size_t)piece * kStateFloats;
                        it.hand = w.handed + piece;
                    }
                } else {
                    // (of a cut chain a copy of it: state_out may be state_in)
                    const int begin = s.from ? plan.chain_begin(piece, s.from) : piece;
                    // (lin_join_kernel's chains: by their last piece)
                    const bool joined = s.from && plan.chain_folds(s) > kMostFolds;
                    if (joined)
                        it.src = w.sum + (size_t)(piece - 1) * kStateFloats;
                    else if (s.to - s.from < s.of && a.state_in && a.state_in == a.state_out)
                        it.src = w.start + (size_t)begin * kStateFloats;
                    else
                        it.src = a.state_in ? a.state_in + chain : nullptr;
                    if (s.from && !joined) it.fold = begin, it.folds = piece - begin;
                }
                if (s.to == s.of && a.state_out) it.dst = a.state_out + chain;
            }
        }
        if (lane == 0) {
            go = mbar_wait(&sh.item_empty[ring], ring_phase ^ 1, 1) ||
                 wait_long(sh, &sh.item_empty[ring], ring_phase ^ 1);
            if (go) {
                sh.item[ring] = it;
                mbar_arrive(&sh.item_full[ring]);
                // (on its way while the last chain is worked on: 64 prompts of 64 tokens, 32
                // heads 123 us, 113)
                if (!SUM && it.src && !it.wait && !it.folds)
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(it.src),
                                 "r"(kStateFloats * 4)
                                 : "memory");
            }
        }
        if (++ring == kRing) ring = 0, ring_phase ^= 1;
        go = __shfl_sync(0xffffffffu, go && it.chunks > 0, 0);
        if (!go) break;
        if (lane == 0) {
            const int hq = a.qk_head(it.h);
            for (int c = 0; go && c < it.chunks; ++c) {
                go = mbar_wait(&sh.empty[stage], phase ^ 1, 1) ||
                     wait_long(sh, &sh.empty[stage], phase ^ 1);
                if (!go) break;
                mbar_arrive_expect_tx(&sh.full[stage], 2 * kTile);
                if (!SUM) mbar_arrive_expect_tx(&sh.v_full[stage], kTile);
                unsigned char* k_tile = sm + (SUM ? stage * kSumStage : stage * kStage + kTile);
                const int row = it.row + c * C;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    unsigned char* dst = k_tile + half * (kTile / 2);
                    if (!SUM)
                        tma_load_3d(dst - kTile, mq, &sh.full[stage], 64 * half, hq, row);
                    tma_load_3d(dst, mk, &sh.full[stage], 64 * half, hq, row);
                }
#pragma unroll
                for (int half = 0; half < 2; ++half)  // (behind Q and K, which are wanted first)
                    tma_load_3d(k_tile + kTile + half * (kTile / 2), mv,
                                SUM ? &sh.full[stage] : &sh.v_full[stage & 1], 64 * half, it.h,
                                row);
                if (++stage == kStages<SUM>) stage = 0, phase ^= 1;
            }
        }
        go = __shfl_sync(0xffffffffu, go, 0);
    }
    // copies in flight must land before the CTA's memory goes away
    if (lane == 0 && *(volatile int*)&sh.stop)
        for (int s = 0; s < kStages<SUM>; ++s)
            mbar_wait(&sh.full[s], s < stage ? phase : phase ^ 1, 1 << 12);
    if (!SUM && lane == 0 && *(volatile int*)&sh.stop)
        for (int s = 0; s < 2; ++s)
            mbar_wait(&sh.v_full[s], s < stage ? phase : phase ^ 1, 1 << 12);
}

// The warp that issues the products: of chunk c P V and Q S, the next chunk's Q K^T, so
// that its weights are worked out while this chunk's W is, and K^T W.  The products of
// one warp run in the order of their issue, so Q K^T may follow P V, over whose P it is
// written.  (In a fixed order: taking whichever has its operands costs more than it
// gains, as the compiler then moves every descriptor into uniform registers again, 66
// cycles a product of 16 k against 130 to 170.)
template <bool F16, bool SUM>
__device__ __forceinline__ void product_role(Shared& sh, unsigned char* sm) {
    constexpr uint32_t kQK = idesc_16(C, C, !F16, false);
    constexpr uint32_t kNT = idesc_16(C, D, !F16, true);   // B as it lies: [K][N]
    constexpr uint32_t kTT = kNT | 1u << 15;               // A too: [K][M]
    constexpr uint64_t kT = kTile >> 4;                    // in a descriptor's units
    const uint32_t tmem = uniform(sh.tmem);
    const uint32_t base = uniform(smem_u32(sm));
    const uint64_t k_major = make_desc_sw128(base, 16);
    const uint64_t mn_major = make_desc_sw128(base, kTile / 2);
    const uint64_t state = mn_major + (kStateTile >> 4);
    auto qk = [&](int stage) {
        const uint64_t q = k_major + stage * (kStage >> 4), k = q + kT;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const uint64_t off = (s >> 2) * (kT / 2) + (s & 3) * 2;
                mma_f16(tmem + kTmemP, q + off, k + off, kQK, s > 0);
            }
            mma_commit(&sh.qk_ready);
        }
        __syncwarp();
    };
    Items items;
    auto next_chunks = [&] {
        const Item* it = items.next(sh);
        const int chunks = it ? it->chunks : 0;
        if (it) items.done(sh);
        return uniform(chunks);
    };
    int left = next_chunks();
    if (left == 0) return;
    if (!SUM) {
        if (!wait_warp(sh, &sh.full[0], 0)) return;
        qk(0);
    }
    int stage = 0;
    for (int n = 0; left > 0; ++n) {
        const uint32_t odd = n & 1, pair = n >> 1 & 1;
        const uint64_t q = k_major + stage * (kStage >> 4);
        const uint64_t k_mn =
            mn_major + (SUM ? stage * (kSumStage >> 4) : stage * (kStage >> 4) + kT);
        const uint64_t v_mn = k_mn + kT, lo_mn = SUM ? state : k_mn - kT;
        if (!SUM) {
            if (n && !wait_warp(sh, &sh.o_read[odd ^ 1], (n - 1) >> 1 & 1)) return;
            if (!wait_warp(sh, &sh.v_checked[odd], pair)) return;
            if (!wait_warp(sh, &sh.p_ready[odd], pair)) return;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_f16_ta(tmem + kTmemPV, tmem + kTmemP + 8 * s, v_mn + s * 128, kNT, s > 0);
                mma_commit(&sh.pv_ready);
                mbar_arrive(&sh.pv_ready);  // passes on what p_ready and v_checked brought
            }
            __syncwarp();
            if (!wait_warp(sh, &sh.s16_ready, odd)) return;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_f16(tmem + kTmemQS, q + (s >> 2) * (kT / 2) + (s & 3) * 2, state + s * 128,
                            kNT, s > 0);
                mma_commit(&sh.qs_ready);
            }
            __syncwarp();
        }
        if (--left == 0) {
            left = next_chunks();
            if (*(volatile int*)&sh.stop) return;
        }
        if (!SUM && left > 0) {
            if (!wait_warp(sh, &sh.full[stage ^ 1], (n + 1) >> 1 & 1)) return;
            qk(stage ^ 1);
        }
        if (!wait_warp(sh, &sh.w_ready[odd], pair)) return;
        tc_fence_after();
        if (elect_one()) {
            // (SUM: two accumulators in turn, as W of the next chunk is ready before this
            // one's product is read; otherwise the last one's was read before S was there)
            const uint32_t to = tmem + (SUM && odd ? kTmemPV : kTmemKW);
#pragma unroll
            for (int s = 0; s < 8; ++s) mma_f16(to, k_mn + s * 128, v_mn + s * 128, kTT, s > 0);
#pragma unroll
            for (int s = 0; s < 8; ++s) mma_f16(to, k_mn + s * 128, lo_mn + s * 128, kTT, true);
            mma_commit(&sh.kw_ready[odd]);
            mma_commit(&sh.empty[stage]);
        }
        __syncwarp();
        if (++stage == kStages<SUM>) stage = 0;
    }
}

// g of a token as it is, 0 for tokens that are not there; and as log2 of the decay.  The
// load is a chunk ahead of its use, and nothing is done with it before.
__device__ __forceinline__ float load_g(const Args& a, const Item& it, int token) {
    return token < it.rows ? __ldg(a.g + ((long long)it.row + token) * a.g_stride + it.h) : 0.f;
}
__device__ __forceinline__ float log2_decay(float g) { return lin::clamp_decay(g) * kLog2e; }

// 16-byte piece `c` (of 8) of row r of a 128-row half tile in the 128-byte swizzle.
__device__ __forceinline__ uint4* piece_of(unsigned char* half_tile, int r, int c) {
    return reinterpret_cast<uint4*>(half_tile + r * 128 + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ void store_32(uint16_t* dst, const uint32_t (&u)[8]) {
    if (reinterpret_cast<uintptr_t>(dst) & 31) {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    } else {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst),
                     "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]),
                     "r"(u[7])
                     : "memory");
    }
}

// Eight floats of a row of a state, a whole sector where the address allows.
__device__ __forceinline__ void load_8(const float* from, float* s) {
    if (reinterpret_cast<uintptr_t>(from) & 31) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(from) + i);
            s[4 * i] = x.x, s[4 * i + 1] = x.y, s[4 * i + 2] = x.z, s[4 * i + 3] = x.w;
        }
    } else {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                     : "=f"(s[0]), "=f"(s[1]), "=f"(s[2]), "=f"(s[3]), "=f"(s[4]), "=f"(s[5]),
                       "=f"(s[6]), "=f"(s[7])
                     : "l"(from)
                     : "memory");
    }
}
__device__ __forceinline__ void store_8(float* to, const float* s) {
    if (reinterpret_cast<uintptr_t>(to) & 31) {
        reinterpret_cast<float4*>(to)[0] = make_float4(s[0], s[1], s[2], s[3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(s[4], s[5], s[6], s[7]);
    } else {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(to),
                     "f"(s[0]), "f"(s[1]), "f"(s[2]), "f"(s[3]), "f"(s[4]), "f"(s[5]), "f"(s[6]),
                     "f"(s[7])
                     : "memory");
    }
}

// The power of two that brings a largest value `x` to [2^13, 2^14) when divided by, and
// its inverse.
__device__ __forceinline__ float unit_of(float x, float& inverse) {
    const int e = min(max((int)(__float_as_uint(x) >> 23) - 13, 1), 241);
    inverse = __uint_as_float((uint32_t)(254 - e) << 23);
    return __uint_as_float((uint32_t)e << 23);
}

// A block of 32 tokens whose decays (log2 of them: g) sum up to so little: differences of its sums
// would lose bits that weights have, 2^-12 of a decay from 4000 on.  Up to here they are good to
// 2^-14.
constexpr float kDeepSum = -256.f;
// Such a block's products on the diagonal, in their place, times the decays: sums of the whole
// parts of g are exact, those of the rest good to 2^-19.  A row a lane; not a path for ordinary
// inputs.
__device__ __noinline__ void deep_decays(uint32_t products, float g) {
    const int lane = threadIdx.x & 31;
    float whole = rintf(g), part = g - whole;
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const float w = __shfl_up_sync(0xffffffffu, whole, off);
        const float p = __shfl_up_sync(0xffffffffu, part, off);
        if (lane >= off) whole += w, part += p;
    }
#pragma unroll 1
    for (int i = 0; i < 32; i += 8) {
        float x[8];
        uint32_t u[8];
        tmem_ld8(products + i, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = (whole - __shfl_sync(0xffffffffu, whole, i + e)) +
                            (part - __shfl_sync(0xffffffffu, part, i + e));
            u[e] = __float_as_uint(i + e <= lane ? x[e] * ex2_approx(d) : 0.f);
        }
        tmem_st8u(products + i, u);
    }
    tmem_st_wait();
}

// Warps 0..3, a thread a token: a chunk's weights P, and the decays that state_role takes
// (SUM: these alone).
template <bool F16, bool SUM>
__device__ __forceinline__ void token_role(const Work& w, Shared& sh, unsigned char* sm) {
    const Args& a = w.a;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const uint32_t row = sh.tmem + ((uint32_t)(warp * 32) << 16);
    Items items;
    int n = 0;
    uint32_t sync_phase = 0;
    while (const Item* const next = items.next(sh)) {
        const Item& it = *next;
        float next_g = load_g(a, it, t);
#pragma unroll 1
        for (int c = 0; c < it.chunks; ++c, ++n) {
            const uint32_t odd = n & 1;
            // (SUM: state_role is through with the last but one chunk's decays)
            if (SUM && n > 1 && !wait_warp(sh, &sh.w_ready[odd], (n - 2) >> 1 & 1)) return;
            const float g = log2_decay(next_g);
            // sums within the block: up to the token, and behind it
            float sum = g, tail = g;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, sum, off);
                const float down = __shfl_down_sync(0xffffffffu, tail, off);
                if (lane >= off) sum += up;
                if (lane + off < 32) tail += down;
            }
            tail = __shfl_down_sync(0xffffffffu, tail, 1);
            if (lane == 31) {
                tail = 0.f;
                sh.block[odd][warp] = sum;
            }
            sh.sum[t] = -sum;
            sh.tail[odd][t] = ex2_approx(tail);
            if (!sync_warps(sh, &sh.token_sync, sync_phase)) return;
            next_g = load_g(a, it, (c + 1) * C + t);
            float before = 0.f, behind = 0.f, total = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = sh.block[odd][i];
                if (i < warp) before += x;
                if (i > warp) behind += x;
                total += x;
            }
            if (lane == 0) sh.later[odd][warp] = ex2_approx(behind);
            if (t == 0) sh.total[odd] = total;
            if (SUM) {
                arrive_warp(&sh.p_ready[odd]);
                continue;
            }

            if (!wait_warp(sh, &sh.qk_ready, odd)) return;
            tc_fence_after();
            // FP16: a row's weights in units that bring its largest product to [2^13, 2^14),
            // or q . k past 65504 would be lost, and so would bits of any below 2^-14.  (Decays
            // make less of a product: weights below 2^-27 of the largest one keep 2^-38 of it.  Eight
            // columns a step, as code here is dear: in steps of 16 16 prompts took 662 us, 644.)
            float inverse = 1.f;
            int unit = 0;
            if (F16) {
                float most = 0.f;
#pragma unroll 1
                for (int i = 0; i < 4 * (warp + 1); ++i) {
                    float x[8];
                    tmem_ld8(row + kTmemP + 8 * i, x);
                    tmem_ld_wait();
                    const int last = t - 8 * i;
#pragma unroll
                    for (int e = 0; e < 8; ++e) most = fmaxf(most, e <= last ? fabsf(x[e]) : 0.f);
                }
                unit = __float_as_uint(unit_of(most, inverse)) >> 23;
            }
            float own = sum;  // of the block on the diagonal
            if (__any_sync(0xffffffffu, sum < kDeepSum)) {
                deep_decays(row + kTmemP + 32 * warp, g);
                sh.sum[t] = own = 0.f;
                __syncwarp();
            }
            // A block of 32 columns a step, upwards: the 16 columns that its weights take
            // hold scores that have been read.  (Rolled: what all roles run has to stay in
            // the instruction cache.)
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                uint32_t p[16] = {};
                if (b <= warp) {
                    float x[32];
                    tmem_ld32(row + kTmemP + 32 * b, x);
                    if (b == warp) {
                        const float4* other = reinterpret_cast<const float4*>(sh.sum + 32 * b);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 s = other[k];
                            float d[4] = {ex2_approx(own + s.x), ex2_approx(own + s.y),
                                          ex2_approx(own + s.z), ex2_approx(own + s.w)};
                            if (F16) {
                                const float2 i2 = make_float2(inverse, inverse);
                                const float2 lo = mul2(make_float2(d[0], d[1]), i2);
                                const float2 hi = mul2(make_float2(d[2], d[3]), i2);
                                d[0] = lo.x, d[1] = lo.y, d[2] = hi.x, d[3] = hi.y;
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[4 * k + e] = 4 * k + e <= lane ? x[4 * k + e] * d[e] : 0.f;
                        }
                    } else {
                        const float4* other =
                            reinterpret_cast<const float4*>(sh.tail[odd] + 32 * b);
                        float from = sum;  // from the end of block b
#pragma unroll 1
                        for (int k = warp - 1; k > b; --k) from += sh.block[odd][k];
                        from = ex2_approx(from);
                        if (F16) from *= inverse;
                        const float2 f2 = make_float2(from, from);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 s = other[k];
                            const float2 lo = mul2(make_float2(x[4 * k], x[4 * k + 1]),
                                                   mul2(make_float2(s.x, s.y), f2));
                            const float2 hi = mul2(make_float2(x[4 * k + 2], x[4 * k + 3]),
                                                   mul2(make_float2(s.z, s.w), f2));
                            x[4 * k] = lo.x, x[4 * k + 1] = lo.y;
                            x[4 * k + 2] = hi.x, x[4 * k + 3] = hi.y;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        p[k] = F16 ? pack_f16x2(x[2 * k], x[2 * k + 1])
                                   : pack_bf16x2(x[2 * k], x[2 * k + 1]);
                }
                tmem_st16u(row + kTmemP + 16 * b, p);
            }
            tmem_st_wait();
            tc_fence_before();
            // The rows behind the last token hold another sequence's: no weight reaches
            // their values, but 0 times infinity would.  V has a barrier of its own: until it
            // has arrived, its copy would write over the zeros.
            const int there = it.rows - c * C;
            if (there < 32 * (warp + 1) && !wait_warp(sh, &sh.v_full[odd], n >> 1 & 1)) return;
            if (t >= there) {
                unsigned char* k_tile = sm + (n & 1) * kStage + kTile;
#pragma unroll 1
                for (int i = 0; i < 32; ++i)  // K's two halves, V's two halves
                    *piece_of(k_tile + (i >> 3) * (kTile / 2), t, i & 7) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            // state_role is through with the last chunk's decays (and P V would wait for
            // the same)
            if (n && !wait_warp(sh, &sh.o_read[odd ^ 1], (n - 1) >> 1 & 1)) return;
            sh.front[t] = ex2_approx(before + sum) * a.scale;
            if (F16) sh.weight_unit[t] = (uint8_t)unit;
            arrive_warp(&sh.p_ready[odd]);
        }
        items.done(sh);
    }
}

// NaN in the columns of half a row of O whose V was not finite at this token or before, in
// global memory or in the half tile on its way there.
template <bool F16>
__device__ __noinline__ void put_nan(uint16_t* o, unsigned char* half_tile,
                                     const uint32_t* bad_first, int half, int t) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
        const int col = 64 * half + i;
        if ((int)(bad_first[col >> 2] >> (col & 3) * 8 & 255u) > t) continue;
        uint16_t* at = o ? o + i
                         : reinterpret_cast<uint16_t*>(piece_of(half_tile, t, i >> 3)) + (i & 7);
        *at = F16 ? 0x7e00 : 0x7fc0;
    }
}

// Looks V over, a warp for half of its columns: what is not finite the product must not see, as
// rows before it have weight 0 for it.  It is set aside as zero, and each column's first such
// row noted: what it does to the rows from there on is put into O and W by state_role.
// (Not a path for ordinary inputs.)  FP16: finds the largest magnitude too.
template <bool F16>
__device__ __noinline__ void set_aside(Shared& sh, unsigned char* half_tile, int half, int r,
                                       int odd) {
    constexpr uint32_t kExp = F16 ? 0x7c00u : 0x7f80u;
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
        uint16_t* at = reinterpret_cast<uint16_t*>(piece_of(half_tile, r, i >> 3)) + (i & 7);
        if ((*at & kExp) != kExp) continue;
        *at = 0;
        const int col = half * 64 + i, shift = (col & 3) * 8;
        uint32_t* word = &sh.bad_first[odd][col >> 2];
        uint32_t was = *(volatile uint32_t*)word;
        while ((was >> shift & 255u) > (uint32_t)r) {
            const uint32_t now = (was & ~(255u << shift)) | (uint32_t)r << shift;
            const uint32_t got = atomicCAS(word, was, now);
            if (got == was) break;
            was = got;
        }
    }
    *(volatile int*)&sh.bad[odd] = 1;
}
template <bool F16>
__device__ __noinline__ void put_back_nan(unsigned char* half_tile, const uint32_t* bad_first,
                                          int half, int r) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
        const int col = half * 64 + i;
        if ((int)(bad_first[col >> 2] >> (col & 3) * 8 & 255u) == r)
            reinterpret_cast<uint16_t*>(piece_of(half_tile, r, i >> 3))[i & 7] =
                F16 ? 0x7e00 : 0x7fc0;
    }
}
// Two FP16 magnitudes: the larger one, at most 65504, as the bits of a float.
__device__ __forceinline__ uint32_t largest_half(uint32_t two) {
    const uint32_t x = min(max(two & 0xffffu, two >> 16), 0x7bffu);
    return __float_as_uint(__half2float(__ushort_as_half((uint16_t)x)));
}
template <bool F16>
__device__ __forceinline__ void check_role(Shared& sh, unsigned char* sm, int half) {
    constexpr uint32_t kExp = F16 ? 0x7c007c00u : 0x7f807f80u,
                       kOne = F16 ? 0x04000400u : 0x00800080u;
    const int lane = threadIdx.x & 31;
    Items items;
    int n = 0;
    while (const Item* const next = items.next(sh)) {
        const Item& it = *next;
#pragma unroll 1
        for (int c = 0; c < it.chunks; ++c, ++n) {
            const uint32_t odd = n & 1;
            const int there = min(C, it.rows - c * C);
            unsigned char* half_tile = sm + (n & 1) * kStage + 2 * kTile + half * (kTile / 2);
            if (!wait_warp(sh, &sh.v_full[n & 1], n >> 1 & 1)) return;
            uint32_t most = 0;
            bool found = false;
#pragma unroll 1
            for (int r = lane; r < C; r += 64) {  // two rows a lane
                uint32_t carry[2] = {0, 0}, largest[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint4 v = *piece_of(half_tile, r + 32 * (i >> 3), i & 7);
                    // an exponent of ones carries into the sign's place
                    carry[i >> 3] |= ((v.x & kExp) + kOne) | ((v.y & kExp) + kOne) |
                                     ((v.z & kExp) + kOne) | ((v.w & kExp) + kOne);
                    if (F16) {
                        uint32_t& m = largest[i >> 3];
                        m = __vmaxu2(__vmaxu2(m, v.x & 0x7fff7fffu),
                                     __vmaxu2(v.y & 0x7fff7fffu, v.z & 0x7fff7fffu));
                        m = __vmaxu2(m, v.w & 0x7fff7fffu);
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const bool mine = r + 32 * k < there;
                    if (F16 && mine) most = __vmaxu2(most, largest[k]);
                    const bool bad = mine && (carry[k] & 0x80008000u);
                    if (__any_sync(0xffffffffu, bad)) {
                        // The last but one chunk's notes are through with once its O is
                        // written, which may be after its V has made room for this one.
                        if (n > 1 && !wait_warp(sh, &sh.o_read[odd], (n - 2) >> 1 & 1)) return;
                        if (bad) set_aside<F16>(sh, half_tile, half, r + 32 * k, odd);
                        found = true;
                    }
                }
            }
            if (F16) {
                const uint32_t m = __reduce_max_sync(0xffffffffu, largest_half(most));
                if (lane == 0) sh.most_v[odd][half] = m;
            }
            if (found) fence_async_smem();
            arrive_warp(&sh.v_checked[odd]);
        }
        items.done(sh);
    }
}

// For a whole warp: until another CTA of the grid has handed its state over, or for at
// most 2^35 clocks.
__device__ __noinline__ bool wait_handed(Shared& sh, const unsigned* flag) {
    const long long from = clock64();
    for (;;) {
        unsigned x;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(x) : "l"(flag) : "memory");
        if (__all_sync(0xffffffffu, x == 1u)) return true;
        bool stop = *(volatile int*)&sh.stop;
        if (!stop && clock64() - from > 1LL << 35) {
            atomicOr(&g_lin_status, STATUS_TIMEOUT);
            *(volatile int*)&sh.stop = 1;
            stop = true;
        }
        if (__any_sync(0xffffffffu, stop)) return false;
        __nanosleep(200);
    }
}

// Warps 4..11, a thread a row i of 64 columns of the state, and likewise a token's 64
// channels of V and O.
template <bool F16, bool SUM>
__device__ __forceinline__ void state_role(const Work& w, Shared& sh, unsigned char* sm,
                                           const CUtensorMap* mo) {
    const Args& a = w.a;
    const int r = threadIdx.x & 127, half = (threadIdx.x >> 7) - 1, warp = r >> 5,
              lane = threadIdx.x & 31, id = (threadIdx.x >> 5) - 4;
    const uint32_t row = sh.tmem + ((uint32_t)(warp * 32) << 16) + 64 * half;
    Items items;
    int n = 0;
    int stage = 0;
    uint32_t state_phase = 0, stage_phase = 0;
    while (const Item* const next = items.next(sh)) {
        const Item& it = *next;
        float s[64];
        {
            const float* from = it.src;
            if (!SUM && it.wait && !wait_handed(sh, it.wait)) return;
            if (!SUM && it.folds) {
                // in the order of memory: a row a thread takes three times as long
                const int at = threadIdx.x - 128;
                float4 x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[i] = from ? __ldcg(reinterpret_cast<const float4*>(from) + at + 256 * i)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                for (int k = it.fold; k < it.fold + it.folds; ++k) {
                    const float d = exp2f(__ldcg(w.log_sum + k));
                    const float4* add =
                        reinterpret_cast<const float4*>(w.sum + (size_t)k * kStateFloats) + at;
#pragma unroll
                    for (int i = 0; i < 16; i += 8) {
                        float4 y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = __ldcg(add + 256 * (i + e));
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x[i + e].x = fmaf(d, x[i + e].x, y[e].x);
                            x[i + e].y = fmaf(d, x[i + e].y, y[e].y);
                            x[i + e].z = fmaf(d, x[i + e].z, y[e].z);
                            x[i + e].w = fmaf(d, x[i + e].w, y[e].w);
                        }
                    }
                }
                float* to = w.folded + (size_t)blockIdx.x * kStateFloats;
#pragma unroll
                for (int i = 0; i < 16; ++i) reinterpret_cast<float4*>(to)[at + 256 * i] = x[i];
                if (!sync_warps(sh, &sh.state_sync, state_phase)) return;
                from = to;
            }
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = 0.f;
            if (from) {
#pragma unroll
                for (int i = 0; i < 8; ++i) load_8(from + r * D + half * 64 + 8 * i, s + 8 * i);
            }
            if (SUM && from) {  // only to be copied
                float* to = w.start + (size_t)blockIdx.x * kStateFloats + r * D + half * 64;
#pragma unroll
                for (int i = 0; i < 8; ++i) store_8(to + 8 * i, s + 8 * i);
#pragma unroll
                for (int i = 0; i < 64; ++i) s[i] = 0.f;
            }
        }
        float decay = 1.f, unit = 1.f, all = 0.f;  // of the last chunk; of the segment
        // the last chunk's part of the state
        auto add = [&] {
            const uint32_t odd = (n - 1) & 1;
            if (!wait_warp(sh, &sh.kw_ready[odd], (n - 1) >> 1 & 1)) return false;
            tc_fence_after();
            const uint32_t at = row + (SUM && odd ? kTmemPV : kTmemKW);
            const float2 d2 = make_float2(decay, decay), u2 = make_float2(unit, unit);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[16];
                tmem_ld16(at + 16 * i, x);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float2 add = make_float2(x[2 * e], x[2 * e + 1]);
                    if (F16) add = mul2(add, u2);
                    const float2 y = fma2(
                        d2, make_float2(s[16 * i + 2 * e], s[16 * i + 2 * e + 1]), add);
                    s[16 * i + 2 * e] = y.x, s[16 * i + 2 * e + 1] = y.y;
                }
            }
            tc_fence_before();
            return true;
        };
#pragma unroll 1
        for (int c = 0; c < it.chunks; ++c, ++n) {
            const uint32_t odd = n & 1;
            const int there = min(C, it.rows - c * C);
            unsigned char* const k_half =
                sm + (SUM ? stage * kSumStage : stage * kStage + kTile) + half * (kTile / 2);
            unsigned char* const v_half = k_half + kTile;
            unsigned char* const state_half = sm + kStateTile + half * (kTile / 2);
            unsigned char* const lo_half = SUM ? state_half : k_half - kTile;
            float f = 0.f, total = 0.f;  // decays from the token on, and of the chunk
            if (SUM) {
                if (!wait_warp(sh, &sh.p_ready[odd], n >> 1 & 1)) return;
                total = sh.total[odd];
                f = sh.tail[odd][r] * sh.later[odd][warp];
            }
            if (SUM && !wait_warp(sh, &sh.full[stage], stage_phase)) return;
            if (++stage == kStages<SUM>) stage = 0, stage_phase ^= 1;
            if (SUM && r >= there) {  // (token_role does it otherwise)
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    *piece_of(k_half, r, i) = make_uint4(0, 0, 0, 0);
                    *piece_of(v_half, r, i) = make_uint4(0, 0, 0, 0);
                }
            }
            if (!SUM && c && !add()) return;
            float v_unit = 1.f, v_inverse = 1.f, s_unit = 1.f, s_inverse = 1.f;
            if (F16) {
                // largest of S (SUM: of V): positive numbers are in order of their bits
                uint32_t most = 0;
                if (SUM) {
                    uint32_t most_v = 0;
#pragma unroll 4
                    for (int i = 0; i < 8; ++i) {
                        const uint4 v = *piece_of(v_half, r, i);
                        most_v = __vmaxu2(__vmaxu2(most_v, v.x & 0x7fff7fffu),
                                          __vmaxu2(v.y & 0x7fff7fffu, v.z & 0x7fff7fffu));
                        most_v = __vmaxu2(most_v, v.w & 0x7fff7fffu);
                    }
                    most = largest_half(most_v);
                } else {
                    float most_s = 0.f;
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        const float x = fabsf(s[i]);
                        most_s = x < INFINITY ? fmaxf(most_s, x) : most_s;
                    }
                    most = __float_as_uint(most_s);
                }
                most = __reduce_max_sync(0xffffffffu, most);
                if (lane == 0) sh.largest[odd][id] = __uint_as_float(most);
                if (!sync_warps(sh, &sh.state_sync, state_phase)) return;
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, sh.largest[odd][i]);
                if (SUM) {
                    v_unit = unit_of(m, v_inverse);
                    f *= v_inverse;
                } else {
                    s_unit = unit_of(m, s_inverse);
                }
            }
            if (!SUM) {
                // (rows of O still on their way from there)
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[8 * i + 2 * e], y = s[8 * i + 2 * e + 1];
                        if (F16) x *= s_inverse, y *= s_inverse;
                        u[e] = narrow2<F16>(x, y);
                    }
                    *piece_of(state_half, r, i) = make_uint4(u[0], u[1], u[2], u[3]);
                }
                fence_async_smem();
                arrive_warp(&sh.s16_ready);
                if (!wait_warp(sh, &sh.pv_ready, odd)) return;  // V is through
                total = sh.total[odd];
                f = sh.tail[odd][r] * sh.later[odd][warp];
                if (F16) {
                    v_unit = unit_of(__uint_as_float(max(sh.most_v[odd][0], sh.most_v[odd][1])),
                                     v_inverse);
                    f *= v_inverse;
                }
            }
            // W: hi over V, then lo over Q (SUM: over the last lo) once that is through
            auto split = [&](int i, uint4& lo) {
                uint4* at = piece_of(v_half, r, i);
                const uint4 v = *at;
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                uint32_t hi[4], rest[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 y = mul2(widen2<F16>(x[e]), make_float2(f, f));
                    hi[e] = narrow2<F16>(y.x, y.y);
                    const float2 h = widen2<F16>(hi[e]);
                    rest[e] = narrow2<F16>(y.x - h.x, y.y - h.y);
                }
                *at = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                lo = make_uint4(rest[0], rest[1], rest[2], rest[3]);
            };
            uint4 lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) split(i, lo[i]);
            if (!SUM) {
                if (*(volatile int*)&sh.bad[odd])
                    put_back_nan<F16>(v_half, sh.bad_first[odd], half, r);
                if (!wait_warp(sh, &sh.qs_ready, odd)) return;
            } else if (c) {  // the last chunk's lo
                if (!wait_warp(sh, &sh.kw_ready[odd ^ 1], (n - 1) >> 1 & 1)) return;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) *piece_of(lo_half, r, i) = lo[i];
            fence_async_smem();
            arrive_warp(&sh.w_ready[odd]);
            if (SUM && c && !add()) return;
            if (!SUM) {
                // the rows of O, while K^T W is under way
                tc_fence_after();
                const float front = sh.front[r] * (F16 ? s_unit : 1.f);
                float scale = a.scale;
                if (F16) scale *= __uint_as_float((uint32_t)sh.weight_unit[r] << 23);
                const float2 d2 = make_float2(front, front), s2 = make_float2(scale, scale);
                // A warp's 32 rows go by way of shared memory, in the place of the state's
                // copy, which Q S is through with (written by the lanes, 32 bytes of a row
                // each, the stores held up everything else on its way to memory: 459 us
                // where this took 447, 16 prompts of 512 to 8192 tokens).  Rows past the
                // last token must not be written: a warp that has some writes its rows
                // itself.
                const bool whole = there >= 32 * (warp + 1);
                const int first = 32 * warp;
                uint16_t* to = a.o + ((long long)it.row + c * C + r) * a.o_stride + it.h * D +
                               64 * half;
#pragma unroll (F16 ? 1 : 2)  // (FP16, 2: 690 us where this took 650, by its longer code)
                for (int i = 0; i < 4; ++i) {  // 16 columns a step
                    float x[16], y[16];
                    tmem_ld16(row + kTmemQS + 16 * i, x);
                    tmem_ld16(row + kTmemPV + 16 * i, y);
                    tmem_ld_wait();
                    uint32_t u[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 o = fma2(d2, make_float2(x[2 * e], x[2 * e + 1]),
                                              mul2(s2, make_float2(y[2 * e], y[2 * e + 1])));
                        u[e] = narrow2<F16>(o.x, o.y);
                    }
                    if (whole) {
                        *piece_of(state_half, r, 2 * i) = make_uint4(u[0], u[1], u[2], u[3]);
                        *piece_of(state_half, r, 2 * i + 1) = make_uint4(u[4], u[5], u[6], u[7]);
                    } else if (r < there) {
                        store_32(to + 16 * i, u);
                    }
                }
                tc_fence_before();
                if (*(volatile int*)&sh.bad[odd]) {
                    if (whole) put_nan<F16>(nullptr, state_half, sh.bad_first[odd], half, r);
                    else if (r < there) put_nan<F16>(to, nullptr, sh.bad_first[odd], half, r);
                    // the last warp cleans up for the chunk after the next one
                    __syncwarp();
                    int seen = 0;
                    if (lane == 0) {
                        __threadfence_block();
                        seen = atomicAdd(&sh.bad_seen[odd], 1);
                        __threadfence_block();
                    }
                    if (__shfl_sync(0xffffffffu, seen, 0) == 7) {
                        sh.bad_first[odd][lane] = 0xffffffffu;
                        if (lane == 0) sh.bad[odd] = sh.bad_seen[odd] = 0;
                    }
                }
                if (whole) fence_async_smem();
                arrive_warp(&sh.o_read[odd]);
                if (whole && lane == 0) {
                    tma_store_3d(mo, state_half + first * 128, 64 * half, it.h,
                                 it.row + c * C + first);
                    bulk_commit();
                }
            }
            decay = ex2_approx(total);
            unit = v_unit;
            all += total;
        }
        if (!add()) return;
        if (it.dst) {
            float* to = it.dst + r * D + half * 64;
#pragma unroll
            for (int i = 0; i < 8; ++i) store_8(to + 8 * i, s + 8 * i);
        }
        if (!SUM && it.hand) {
            if (!sync_warps(sh, &sh.state_sync, state_phase)) return;
            if (threadIdx.x == 128) {
                __threadfence();
                asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(it.hand), "r"(1u)
                             : "memory");
            }
        }
        if (SUM && r == 0 && half == 0) w.log_sum[blockIdx.x] = all;
        items.done(sh);
    }
}

template <bool F16, bool SUM>
__global__ void __launch_bounds__(kThreads, 1)
lin_prefill_kernel(Work w, const __grid_constant__ CUtensorMap mq,
                   const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv,
                   const __grid_constant__ CUtensorMap mo) {
    extern __shared__ __align__(1024) unsigned char sm[];
    Shared& sh = *reinterpret_cast<Shared*>(sm + kSharedOff);
    const int warp = threadIdx.x >> 5;
    if (smem_u32(sm) & 1023u) {  // the swizzle goes by address bits
        if (threadIdx.x == 0) atomicOr(&g_lin_status, STATUS_SMEM_ALIGN);
        return;
    }
    if (threadIdx.x == 0) {
        sh.stop = 0;
        for (int i = 0; i < 3; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sh.v_full[i], 1), sh.bad[i] = sh.bad_seen[i] = 0;
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], SUM ? 13 : 15);
        }
        mbar_init(&sh.qk_ready, 1);
        mbar_init(&sh.pv_ready, 2);
        mbar_init(&sh.s16_ready, 8);
        mbar_init(&sh.qs_ready, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.p_ready[i], 4);
            mbar_init(&sh.v_checked[i], 2);
            mbar_init(&sh.w_ready[i], 8);
            mbar_init(&sh.kw_ready[i], 1);
            mbar_init(&sh.o_read[i], 8);
        }
        mbar_init(&sh.token_sync, 4);
        mbar_init(&sh.state_sync, 8);
        fence_mbar_init();
        prefetch_tmap(&mq);
        prefetch_tmap(&mk);
        prefetch_tmap(&mv);
        if (!SUM) prefetch_tmap(&mo);
    }
    if (threadIdx.x < 2 * (D / 4)) (&sh.bad_first[0][0])[threadIdx.x] = 0xffffffffu;
    if (warp == 13) tmem_alloc(&sh.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    if (SUM && threadIdx.x == 0) w.handed[blockIdx.x] = 0;
    if (warp == 12) {
        copy_role<SUM>(w, sh, sm, &mq, &mk, &mv);
    } else if (warp == 13) {
        product_role<F16, SUM>(sh, sm);
    } else if (warp >= 4 && warp < 12) {
        state_role<F16, SUM>(w, sh, sm, &mo);
        if (!SUM) bulk_wait_all();  // rows of O on their way (lane 0's)
    } else if (warp < 4) {
        token_role<F16, SUM>(w, sh, sm);
    } else if (!SUM) {
        check_role<F16>(sh, sm, warp - 14);
    }
    if (!SUM && warp == 15 && w.a.cu) {
        const Args& a = w.a;
        const int lane = threadIdx.x & 31;
        if (blockIdx.x == 0 && !warp_offsets_ok(a.cu, a.n_seqs, a.t) && lane == 0)
            atomicOr(&g_lin_status, STATUS_BAD_CU_SEQLENS);
        // states of sequences without tokens
        for (int n0 = 0; a.state_out && a.state_out != a.state_in && n0 < a.n_seqs; n0 += 32) {
            lin::Rows rows;
            unsigned empty = __ballot_sync(0xffffffffu, n0 + lane < a.n_seqs &&
                                                            sequence_rows(a, n0 + lane, rows) &&
                                                            rows.count == 0);
            for (; empty; empty &= empty - 1) {
                const long long chain = (long long)(n0 + __ffs(empty) - 1) * a.heads;
                for (int h = 0; h < a.heads; ++h) {
                    if ((chain + h) % gridDim.x != blockIdx.x) continue;
                    const size_t at = (size_t)(chain + h) * kStateFloats;
                    for (int i = lane; i < kStateFloats / 4; i += 32)
                        reinterpret_cast<float4*>(a.state_out + at)[i] =
                            a.state_in ? reinterpret_cast<const float4*>(a.state_in + at)[i]
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 13) tmem_dealloc(sh.tmem, 512);
}

// States in front of the parts of chains that are cut: from each chain's beginning, S
// <- 2^log_sum S + sum through its pieces.  Four floats a thread.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) lin_join_kernel(Work w) {
    const Args& a = w.a;
    pdl_wait();
    pdl_release();
    const Plan p = make_plan(w);
    const int i = blockIdx.x;
    Segment s;
    if (!open_segment(w, p, i, s) || s.from || p.chain_folds(s) <= kMostFolds) return;
    // pieces whose last segment is this chain's and open
    int last = i + padded(s.of, p.piece) - 2;
    if (p.kind == kEven) {
        const long long chain_end = (long long)(i + 1) * p.piece + (s.of - s.to);
        last = (int)((chain_end - 1) / p.piece) - 1;
    }
    const int at = blockIdx.y * kJoinThreads + threadIdx.x;  // of the state's float4s
    const size_t chain = ((size_t)s.n * a.heads + s.h) * kStateFloats;
    float4 x = a.state_in ? __ldcg(reinterpret_cast<const float4*>(a.state_in + chain) + at)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    float4* sums = reinterpret_cast<float4*>(w.sum) + at;
    // (eight loads in flight: a load may not pass the stores before it by itself)
    constexpr int kBatch = 8;
    for (int k0 = i; k0 <= last; k0 += kBatch) {
        float4 add[kBatch];
        float d[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (k0 + k > last) break;
            add[k] = __ldcg(sums + (size_t)(k0 + k) * (kStateFloats / 4));
            d[k] = __ldcg(w.log_sum + k0 + k);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (k0 + k > last) break;
            const float by = exp2f(d[k]);
            x.x = fmaf(by, x.x, add[k].x);
            x.y = fmaf(by, x.y, add[k].y);
            x.z = fmaf(by, x.z, add[k].z);
            x.w = fmaf(by, x.w, add[k].w);
            sums[(size_t)(k0 + k) * (kStateFloats / 4)] = x;
        }
    }
}

// Pieces that a call has at most.
int most_pieces(long long rows, int n_seqs, int heads) {
    return (int)std::min<long long>(kSms, (rows / C + n_seqs) * heads);
}

}  // namespace

cudaError_t status_word_lin(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_lin_status);
}

size_t lin_chunked_workspace_bytes(long long rows, int n_seqs, int heads) {
    return (size_t)most_pieces(rows, n_seqs, heads) * (3 * kStateFloats + 8) * sizeof(float);
}

kda_status launch_lin_chunked(const Args& a, bool f16, void* workspace, cudaStream_t s) {
    const char* fn = "kda_lin_prefill";
    const long long rows = a.cu ? a.t : (long long)a.t_pad * a.n_seqs;
    const int sms = sm_count();
    KDA_REQUIRE(sms > 0, KDA_ERR_CUDA, "%s: no device", fn);
    Work w = {a};
    const int slots = most_pieces(rows, a.n_seqs, a.heads);
    w.pieces = std::min(slots, sms);
    w.sum = static_cast<float*>(workspace);
    w.start = w.sum + (size_t)slots * kStateFloats;
    w.folded = w.start + (size_t)slots * kStateFloats;
    w.log_sum = w.folded + (size_t)slots * kStateFloats;
    w.handed = reinterpret_cast<unsigned*>(w.log_sum + 4 * (size_t)slots);
    CUtensorMap mq, mk, mv, mo;
    KDA_REQUIRE(tma_map_heads(&mq, a.q, a.qk_heads, rows, a.q_stride, 1, C, f16) &&
                    tma_map_heads(&mk, a.k, a.qk_heads, rows, a.k_stride, 1, C, f16) &&
                    tma_map_heads(&mv, a.v, a.heads, rows, a.v_stride, 1, C, f16) &&
                    tma_map_heads(&mo, a.o, a.heads, rows, a.o_stride, 1, 32, f16),
                KDA_ERR_CUDA, "%s: cannot describe the arrays to the copy engine", fn);
    // Whether sums may be wanted, and whether states may be handed over between CTAs: for
    // packed rows the lengths are on the device.
    const long long chains = (long long)a.n_seqs * a.heads;
    const long long longest = (a.t + C - 1) / C;
    const bool whole = longest <= kWhole && chains <= w.pieces;
    w.least = whole ? kWhole : kLeastPiece;
    const long long pads = (longest + w.least - 1) / w.least;
    const bool few = pads * chains <= w.pieces;
    const long long piece =
        few ? w.least
            : std::max<long long>(((longest + kLead) * chains + w.pieces - 1) / w.pieces, w.least);
    bool cut, hand;
    int grid = w.pieces;
    if (a.cu) {
        cut = hand = !whole;
    } else if (few && (pads == 1 || !hand_over(longest, piece))) {
        cut = pads > 1;
        hand = false;
        grid = (int)(pads * chains);
    } else {
        hand = hand_over(longest, piece);
        cut = !hand;
    }
    // (a piece has at least a share of the longest sequence's chunks)
    const long long least = std::max<long long>(w.least, longest * a.heads / w.pieces);
    const bool join = longest / least + 1 > kMostFolds;
    auto kernel = f16 ? lin_prefill_kernel<true, false> : lin_prefill_kernel<false, false>;
    auto sums = f16 ? lin_prefill_kernel<true, true> : lin_prefill_kernel<false, true>;
    for (auto k : {kernel, sums}) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)kSmemBytes);
        if (e != cudaSuccess) {
            set_error("%s: cannot reserve shared memory: %s", fn, cudaGetErrorString(e));
            return KDA_ERR_CUDA;
        }
    }
    if (cut) {
        launch_pdl(sums, dim3(grid), dim3(kThreads), kSmemBytes, s, w, mq, mk, mv, mo);
        if (join)
            launch_pdl(lin_join_kernel, dim3(grid, kStateFloats / 4 / kJoinThreads),
                       dim3(kJoinThreads), 0, s, w);
    } else if (hand) {
        cudaMemsetAsync(w.handed, 0, slots * sizeof(unsigned), s);
    }
    if (!hand) {
        launch_pdl(kernel, dim3(grid), dim3(kThreads), kSmemBytes, s, w, mq, mk, mv, mo);
        return launch_result(fn);
    }
    // CTAs that may wait for one another run together
    void* args[] = {&w, &mq, &mk, &mv, &mo};
    cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(kThreads),
                                args, kSmemBytes, s);
    return launch_result(fn);
}

}  // namespace kda
