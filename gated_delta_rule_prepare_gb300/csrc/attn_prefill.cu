// Causal attention of packed prompts (kda_attn_prefill).  For query row i of a
// sequence of Lq queries and Lk keys, at position p = Lk - Lq + i, head h and
// its KV head h / (heads / kv_heads):
//     s_j = scale * q_i . k_j          for max(0, p - window + 1) <= j <= p
//     o_i = sum_j exp(s_j - lse) v_j,  lse = log sum_j exp(s_j)
// A row that sees no key gives o = 0 and lse = -inf.
//
// Bound by the tensor cores: 512 FLOP per (query row, key) against 512 bytes
// per key and tile.  The shape of the work:
//  - A tile is 128 rows of Q: the G = heads / kv_heads query heads of one KV
//    head for 128 / G consecutive tokens (rows past G * (128 / G) idle).  The
//    heads that share keys share their loads, and a tile spans few tokens, so
//    little of its last key block is masked.
//  - A work item is two such tiles, one after the other in the sequence, and
//    walks their keys in blocks of 128.  S = Q K^T (FP32) sits in TMEM, one
//    thread owns one row of it, and writes exp2(S - shift) over it in 16 bits,
//    from where the second product reads it as its A operand.  The tensor
//    cores work for one tile while the other tile's softmax runs.
//  - One persistent CTA per SM: a TMA warp, a warp for each tile that issues its
//    MMAs, four softmax warps for each tile, four warps that write finished
//    tiles, so the next item's first block overlaps the last one's end.
//  - Items go out by a ticket counter in the order that attn_plan_kernel writes;
//    a call whose items fit one per SM needs neither.  Where items are few, or a
//    chunk's do not fill the last round, CTAs share an item's keys.
//  - The roles' loops are kept short, and what is rare out of them: they meet in
//    one instruction cache.
// BF16, 32 heads over 8: 1707 TFLOP/s at 8192 tokens, 1859 at 32768, 1682 at 16
// packed prompts of 512 to 8192 (cuBLAS's 8192^3 product: 1940), each a burst of a
// few calls.  Called for seconds, at the power limit, those prompts run at 1510 to
// 1540 (cuBLAS 1714).  What is left is an item's start and end, a part of a round
// when items do not fill the SMs evenly, and the issue of the softmax.
#include <algorithm>
#include <cmath>

#include "attn_common.h"
#include "f32x2.h"
#include "sm103_tc.h"
#include "tma_map.h"

namespace kda {
namespace {

using namespace attn;
using namespace tc;

__device__ unsigned g_attn_status = 0;

struct Redo;
struct PrefillArgs {
    const uint16_t *q, *k, *v;
    uint16_t* o;
    float* lse;
    const int *cu_q, *cu_k;
    long long q_stride, k_stride, v_stride, o_stride;
    int t_q, t_k, n_seqs, heads, kv_heads, window;
    int group, tile_tokens;  // heads per KV head; tokens per tile
    float scale;
    int4* list;       // ordered entries; null: one sequence's, or one item per CTA
    bool one;         // sequence: its entries need no list, its items no counter
    int4* group_of;   // of an entry: its sequence's first entry, their number, KV heads at a time
    int* first_entry; // of a sequence
    unsigned* count;  // entries in the list, then the ticket counter
    Redo* redo;  // [item][tile][warp]
    int slots, bucket_shift;
    // Items from `shared` on have their keys cut into `splits` shares, without a list
    // one CTA each, with one a ticket each.
    int splits, shared;
    float* part;         // their outputs [item - shared][share][256 rows][128], unscaled
    float2* part_stat;   // and (shift, sum) of their rows
};

// Sequence n's query and key rows; false for offsets outside the arrays.
struct Span {
    int q0, k0, lq, lk;
};
__device__ __forceinline__ bool sequence_span(const PrefillArgs& a, int n, Span& s) {
    if (!a.cu_q) {
        s = {n * a.t_q, n * a.t_k, a.t_q, a.t_k};
        return true;
    }
    const int q0 = __ldg(a.cu_q + n), q1 = __ldg(a.cu_q + n + 1);
    const int k0 = __ldg(a.cu_k + n), k1 = __ldg(a.cu_k + n + 1);
    s = {q0, k0, q1 - q0, k1 - k0};
    return q0 >= 0 && q0 <= q1 && q1 <= a.t_q && k0 >= 0 && k0 <= k1 && k1 <= a.t_k;
}

// An item's tokens, all heads: first query row, tokens (at most two tiles'),
// first key row of the sequence, position of the first token (it may be
// negative).  Keys of the sequence end at its last query's position.
struct Entry {
    int row, tokens, k0, pos;
};

// 32 rows of a tile, some of them (bits of `rows`) to be done again, and the
// record of the same CTA before it.  One place per item, tile and warp.
struct Redo {
    Entry e;
    int head;
    unsigned rows;
    int before;
};

// Slots number the items of all sequences: sequence n, whose queries start at
// row c, owns slots from c / span + n (span = 2 tiles of tokens), never fewer
// than it has items.
__device__ __forceinline__ long long first_slot(const PrefillArgs& a, int n) {
    const int span = 2 * a.tile_tokens;
    const long long c = a.cu_q ? (long long)__ldg(a.cu_q + n) : (long long)n * a.t_q;
    return c / span + n;
}
__device__ __forceinline__ bool slot_entry(const PrefillArgs& a, int n, long long slot, Entry& e) {
    Span s;
    if (!sequence_span(a, n, s)) return false;
    const int span = 2 * a.tile_tokens;
    const long long i = (slot - first_slot(a, n)) * span;  // first token
    if (i < 0 || i >= s.lq) return false;
    e = {s.q0 + (int)i, min(span, s.lq - (int)i), s.k0, s.lk - s.lq + (int)i};
    return true;
}

// The first key that a query at position `pos` sees (below 0: it sees none), window
// 0 for no window; windows up to 2^31 - 1 are taken.
__device__ __forceinline__ int first_seen(int pos, int window) {
    return window ? max(0, max(pos, -1) + 1 - window) : 0;
}

// Key blocks [lo, hi) of 128 that `tokens` tokens from position `pos` see.
__device__ __forceinline__ void key_blocks(const PrefillArgs& a, int pos, int tokens, int& lo,
                                           int& hi) {
    const int last = pos + tokens - 1;
    lo = first_seen(pos, a.window) >> 7;
    hi = tokens > 0 && last >= 0 ? (last >> 7) + 1 : lo;
    if (hi < lo) hi = lo;
}

// Writes the entries in the order in which they are worked on, and zeroes the
// ticket counter: sequences with the most keys first (a counting sort), of each
// its last tokens first.  Items are a sequence's entries for as many KV heads as
// have kL2Bytes of keys and values, heads innermost, then for the next ones: what
// runs at a time reads what the L2 cache holds, and the last items are short.
// (Entries of all sequences sorted together: 2187 us at the front end's 16
// prompts, whose keys and values are 360 MB; a head at a time: 1854, but 358
// instead of 346 for one of 8192 tokens, whose last head then keeps few CTAs.)
// One CTA; at those prompts it writes about 1400 entries.
constexpr int kL2Bytes = 48 << 20;
__device__ __forceinline__ int heads_at_a_time(int lk) {
    return max(1, kL2Bytes / (4 * D) / max(1, lk));
}
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(PrefillArgs a) {
    __shared__ int hist[kPlanThreads];
    __shared__ int warp_sum[32];
    pdl_wait();
    pdl_release();
    __shared__ bool overlap;
    const int tid = threadIdx.x, span = 2 * a.tile_tokens;
    hist[tid] = 0;
    if (tid < 32) {
        const bool ok = !a.cu_q || (warp_offsets_ok(a.cu_q, a.n_seqs, a.t_q) &&
                                    warp_offsets_ok(a.cu_k, a.n_seqs, a.t_k));
        const bool slots_ok = ok || warp_offsets_rise(a.cu_q, a.n_seqs, a.t_q);
        if (tid == 0) {
            overlap = !slots_ok;
            if (!ok) atomicOr(&g_attn_status, STATUS_BAD_CU_SEQLENS);
        }
    }
    __syncthreads();
    // Query offsets that fall or leave the array: sequences may overlap, have more
    // entries than there are slots, and slots that name others.  Nothing is done.
    if (overlap) {
        if (tid < 2) a.count[tid] = 0;
        return;
    }
    // bucket 0 holds the longest sequences
    auto sequence = [&](int n, int& bucket) {
        Span s;
        if (!sequence_span(a, n, s)) return 0;
        bucket = kPlanThreads - 1 - min(s.lk >> (7 + a.bucket_shift), kPlanThreads - 1);
        return (s.lq + span - 1) / span;
    };
    int bucket = 0;
    for (int n = tid; n < a.n_seqs; n += kPlanThreads) {
        const int entries = sequence(n, bucket);
        if (entries) atomicAdd(&hist[bucket], entries);
    }
    __syncthreads();
    const int mine = hist[tid];
    int sum = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, off);
        if ((tid & 31) >= off) sum += up;
    }
    if ((tid & 31) == 31) warp_sum[tid >> 5] = sum;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < (tid >> 5); ++w) before += warp_sum[w];
    hist[tid] = before + sum - mine;
    if (tid == kPlanThreads - 1) {
        a.count[0] = before + sum;
        a.count[1] = 0;
    }
    __syncthreads();
    for (int n = tid; n < a.n_seqs; n += kPlanThreads) {
        const int entries = sequence(n, bucket);
        a.first_entry[n] = entries ? atomicAdd(&hist[bucket], entries) : 0;
    }
    __syncthreads();
    for (int slot = tid; slot < a.slots; slot += kPlanThreads) {
        int n = 0, left = a.n_seqs;
        while (left > 1) {
            const int half = left / 2;
            if (first_slot(a, n + half) <= slot) {
                n += half;
                left -= half;
            } else {
                left = half;
            }
        }
        Entry e;
        if (!slot_entry(a, n, slot, e)) continue;
        const int base = a.first_entry[n], entries = sequence(n, bucket);
        const int at = base + entries - 1 - (int)(slot - first_slot(a, n));
        a.list[at] = make_int4(e.row, e.tokens, e.k0, e.pos);
        Span whole;
        sequence_span(a, n, whole);
        a.group_of[at] = make_int4(base, entries, heads_at_a_time(whole.lk), 0);
    }
}

// One row on the CUDA cores by one warp, 4 channels a lane, touching only the
// keys that the row sees.  The tensor cores multiply a masked key's weight 0
// with its value, which gives NaN where the value is infinite or NaN; rows that
// come out so are done again here, and rows whose weights left FP32's range
// (softmax_role).  Not a path for ordinary inputs.
template <bool F16>
__device__ __noinline__ void attend_row(const PrefillArgs& a, long long row, long long k0, int p,
                                        int h) {
    const int lane = threadIdx.x & 31;
    const int hk = h / a.group;
    const int first = first_seen(p, a.window);
    const uint2 qb = __ldg(reinterpret_cast<const uint2*>(a.q + row * a.q_stride + h * D +
                                                          4 * lane));
    const float c = a.scale * kLog2e;
    const float2 q01 = widen2<F16>(qb.x), q23 = widen2<F16>(qb.y);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const uint16_t* kp = a.k + k0 * a.k_stride + hk * D + 4 * lane;
    const uint16_t* vp = a.v + k0 * a.v_stride + hk * D + 4 * lane;
#pragma unroll 1
    for (int j = first; j <= p; ++j) {
        const uint2 kb = __ldg(reinterpret_cast<const uint2*>(kp + j * a.k_stride));
        const uint2 vb = __ldg(reinterpret_cast<const uint2*>(vp + j * a.v_stride));
        const float2 k01 = widen2<F16>(kb.x), k23 = widen2<F16>(kb.y);
        float d = q01.x * k01.x;
        d = fmaf(q01.y, k01.y, d);
        d = fmaf(q23.x, k23.x, d);
        d = fmaf(q23.y, k23.y, d);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        d *= c;
        const float m2 = fmaxf(m, d);
        const float shift = m2 == -INFINITY ? 0.f : m2;
        const float keep = exp2f(m - shift), w = exp2f(d - shift);
        const float2 v01 = widen2<F16>(vb.x), v23 = widen2<F16>(vb.y);
        l = fmaf(l, keep, w);
        o.x = fmaf(o.x, keep, w * v01.x);
        o.y = fmaf(o.y, keep, w * v01.y);
        o.z = fmaf(o.z, keep, w * v23.x);
        o.w = fmaf(o.w, keep, w * v23.y);
        m = m2;
    }
    const float r = l == 0.f ? 0.f : 1.f / l;
    const uint2 out = make_uint2(narrow2<F16>(o.x * r, o.y * r), narrow2<F16>(o.z * r, o.w * r));
    *reinterpret_cast<uint2*>(a.o + row * a.o_stride + h * D + 4 * lane) = out;
    if (a.lse && lane == 0)
        a.lse[row * a.heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- the kernel
constexpr int kThreads = 512;
constexpr int kStages = 5;                 // of 32 KB: a block's K, then its V
constexpr uint32_t kTileBytes = 128 * 128 * 2;
constexpr int kRing = 4;                   // items between the TMA warp and the others
constexpr uint32_t kTmemO = 256;           // S0, S1, O0, O1: 128 columns each
// The softmax's thresholds: see softmax_role.
constexpr float kLag = 16777216.f;  // 2^24
template <bool F16>
constexpr float kLift = F16 ? 7.f : 0.f;

struct Item {
    Entry e;
    int head;      // KV head; negative: no more items
    int index;     // of all the call's items; of a share, -1 less its part's number
    int from, to;  // key blocks of it that this CTA has
};

struct Shared {
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2][2];  // P: keys 0..63 of the block, keys 64..127
    uint64_t turn[2];
    uint64_t o_full[2], o_empty[2], sum_full[2];
    uint64_t item_full[kRing], item_empty[kRing];
    Item item[kRing];
    float sum[2][128];   // finished rows' sums of weights
    uint32_t tmem;
    int stop;  // a wait gave up: everybody leaves
    int redo;  // this CTA's last record of rows to be done again, or -1
};
constexpr uint32_t kSharedOff = (2 + kStages) * kTileBytes;
constexpr uint32_t kSmemBytes = kSharedOff + sizeof(Shared);
static_assert(kSmemBytes <= 232448, "shared memory");

// Waits with an end: a phase that does not come within 2^35 clocks (some 17
// seconds), or another role's giving up, ends the kernel with an error status.
// (Rows are done again after all waits.)  The long wait
// is a function of its own: between the roles' loops its code costs room in the
// instruction cache (8192 tokens, 32 heads over 8: 331 us with it there, 320).
__device__ __noinline__ bool wait_long(Shared& sh, uint64_t* bar, uint32_t parity) {
    const long long from = clock64();
    while (!mbar_wait(bar, parity, 32)) {
        if (*(volatile int*)&sh.stop) return false;
        if (clock64() - from > 1LL << 35) {
            atomicOr(&g_attn_status, STATUS_TIMEOUT);
            *(volatile int*)&sh.stop = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity) {
    return mbar_wait(bar, parity, 1) || wait_long(sh, bar, parity);
}
// For a whole warp, which leaves together.
__device__ __forceinline__ bool wait_warp(Shared& sh, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(sh, bar, parity));
}

// Tile t's tokens and key blocks within an item.
struct Tile {
    int tokens, pos, lo, hi;
};
__device__ __forceinline__ Tile tile_of(const PrefillArgs& a, const Item& it, int t) {
    Tile r;
    r.tokens = min(a.tile_tokens, it.e.tokens - t * a.tile_tokens);
    if (r.tokens < 0) r.tokens = 0;
    r.pos = it.e.pos + t * a.tile_tokens;
    key_blocks(a, r.pos, r.tokens, r.lo, r.hi);
    r.lo = max(r.lo, it.from);
    r.hi = max(r.lo, min(r.hi, it.to));
    return r;
}
// The union of both tiles' blocks (their ranges overlap or touch).
struct Blocks {
    int lo, hi;
};
__device__ __forceinline__ Blocks blocks_of(const Tile& x, const Tile& y) {
    if (x.hi <= x.lo) return {y.lo, y.hi};
    if (y.hi <= y.lo) return {x.lo, x.hi};
    return {min(x.lo, y.lo), max(x.hi, y.hi)};
}

// Entries in order.
__device__ __forceinline__ int one_entries(const PrefillArgs& a) {
    Span s;
    if (!sequence_span(a, 0, s)) return 0;
    return (s.lq + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
}
__device__ __forceinline__ int entry_count(const PrefillArgs& a) {
    return a.list ? (int)__ldcg(a.count) : a.one ? one_entries(a) : 0;
}
// Item x in order, whole.
__device__ __forceinline__ void ordered_item(const PrefillArgs& a, unsigned x, Item& it) {
    // any entry of the item's sequence, then the item's
    int4 seq;
    if (a.list) {
        seq = __ldcg(a.group_of + x / (unsigned)a.kv_heads);
    } else {
        Span s;
        sequence_span(a, 0, s);
        seq = make_int4(0, one_entries(a), heads_at_a_time(s.lk), 0);
    }
    int i = (int)(x - (unsigned)seq.x * a.kv_heads);
    const int heads = min(seq.z, a.kv_heads);  // of a full group
    const int group = i / (seq.y * heads), first = group * heads;
    i -= group * seq.y * heads;
    const int here = min(heads, a.kv_heads - first);
    it.head = first + i % here;
    if (a.list) {
        const int4 v = __ldcg(a.list + seq.x + i / here);
        it.e = {v.x, v.y, v.z, v.w};
    } else {
        slot_entry(a, 0, first_slot(a, 0) + seq.y - 1 - i / here, it.e);
    }
    it.index = (int)x;
}
__device__ __forceinline__ void take_share(const PrefillArgs& a, Item& it, int share) {
    const Blocks b = blocks_of(tile_of(a, it, 0), tile_of(a, it, 1));
    const int each = (b.hi - b.lo + a.splits - 1) / a.splits;
    it.from = b.lo + share * each;
    it.to = it.from + each;
    it.index = -1 - ((it.index - a.shared) * a.splits + share);
}

// The TMA warp: hands out items and fills the Q tiles and the ring of K and V.
template <bool CUT>
__device__ __forceinline__ void load_role(const PrefillArgs& a, Shared& sh, unsigned char* sm,
                                          const CUtensorMap* mq, const CUtensorMap* mk,
                                          const CUtensorMap* mv) {
    const int lane = threadIdx.x & 31;
    int stage = 0;
    uint32_t phase = 0, q_phase[2] = {0, 0}, ring_phase = 0;
    int ring = 0;
    const unsigned n_items = (unsigned)entry_count(a) * a.kv_heads;
    bool go = true;
    for (int round = 0; go; ++round) {
        Item it;
        it.head = -1;
        it.from = 0;
        it.to = 0x7fffffff;
        if (a.list || a.one) {
            unsigned x;
            if (a.list) {
                if (lane == 0) x = atomicAdd(a.count + 1, 1u);
                x = __shfl_sync(0xffffffffu, x, 0);
            } else {
                // there and back, as the items get shorter
                x = round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            }
            // shares of the last items: first of all the first ones, so that keys
            // in use at a time are few
            unsigned share = 0;
            const bool cut = CUT && x >= (unsigned)a.shared;
            if (cut && n_items > (unsigned)a.shared) {
                const unsigned n_shared = n_items - a.shared;
                share = (x - a.shared) / n_shared;
                x = share < (unsigned)a.splits ? a.shared + (x - a.shared) % n_shared : n_items;
            }
            if (x < n_items) {
                ordered_item(a, x, it);
                if (cut) take_share(a, it, (int)share);
            }
        } else if (round == 0) {
            it.index = CUT ? blockIdx.x / a.splits : blockIdx.x;
            const int slot = it.index / a.kv_heads;
            const int split = CUT ? blockIdx.x - it.index * a.splits : 0;
            const int n = warp_find_last(a.n_seqs, slot, [&](int i) { return first_slot(a, i); });
            if (slot_entry(a, n, slot, it.e)) {
                it.head = it.index - slot * a.kv_heads;
                if (CUT) take_share(a, it, split);
            }
        }
        if (lane == 0) {
            go = wait(sh, &sh.item_empty[ring], ring_phase ^ 1);
            if (go) {
                sh.item[ring] = it;
                mbar_arrive(&sh.item_full[ring]);
            }
        }
        if (++ring == kRing) ring = 0, ring_phase ^= 1;
        go = __shfl_sync(0xffffffffu, go && it.head >= 0, 0);
        if (!go) break;
        if (lane == 0) {
            const Tile tile[2] = {tile_of(a, it, 0), tile_of(a, it, 1)};
            const uint32_t q_bytes = (uint32_t)(a.group * a.tile_tokens) * 256;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (!go || tile[t].hi <= tile[t].lo) continue;
                go = wait(sh, &sh.q_empty[t], q_phase[t] ^ 1);
                q_phase[t] ^= 1;
                if (!go) continue;
                mbar_arrive_expect_tx(&sh.q_full[t], q_bytes);
                for (int half = 0; half < 2; ++half)
                    tma_load_3d(sm + t * kTileBytes + half * (kTileBytes / 2), mq, &sh.q_full[t],
                                64 * half, it.head * a.group, it.e.row + t * a.tile_tokens);
            }
            const Blocks b = blocks_of(tile[0], tile[1]);
            for (int j = b.lo; go && j < b.hi; ++j) {
                for (int which = 0; which < 2; ++which) {
                    go = go && wait(sh, &sh.kv_empty[stage], phase ^ 1);
                    if (!go) break;
                    mbar_arrive_expect_tx(&sh.kv_full[stage], kTileBytes);
                    unsigned char* dst = sm + (2 + stage) * kTileBytes;
                    for (int half = 0; half < 2; ++half)
                        tma_load_3d(dst + half * (kTileBytes / 2), which ? mv : mk,
                                    &sh.kv_full[stage], 64 * half, it.head, it.e.k0 + j * 128);
                    if (++stage == kStages) stage = 0, phase ^= 1;
                }
            }
        }
        go = __shfl_sync(0xffffffffu, go, 0);
    }
    // copies in flight must land before the CTA's memory goes away: each stage
    // that was filled and not waited for
    if (lane == 0 && *(volatile int*)&sh.stop) {
        for (int s = 0; s < kStages; ++s)
            mbar_wait(&sh.kv_full[s], s < stage ? phase : phase ^ 1, 1 << 12);
        for (int t = 0; t < 2; ++t) mbar_wait(&sh.q_full[t], q_phase[t] ^ 1, 1 << 12);
    }
}

// One lane of the warp, always the same one.  The issuing warp runs its code
// together and only the MMAs and commits are the elected lane's, so that
// descriptors stay in uniform registers (from a branch of lane 0 alone each was
// moved there again).
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(yes));
    return yes != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// The warp that issues tile t's MMAs: per block S = Q K^T, and O += P V once
// the softmax has written P.  Each tile has a warp of its own, so that the
// waits of one tile's products run under the other's; they take turns, so that
// one tile's products run while the other's softmax does (one warp for both:
// 1366 TFLOP/s at 8192 tokens, 32 heads over 8; two without turns: 1279; with:
// 1424, before the softmax was shortened).  MMAs of one warp execute in the
// order of their issue, so S's write over P needs no wait of its own.
template <bool F16, int t>
__device__ __forceinline__ void mma_role(const PrefillArgs& a, Shared& sh, unsigned char* sm) {
    constexpr uint32_t kQK = idesc_16(128, 128, !F16, false);
    constexpr uint32_t kPV = idesc_16(128, 128, !F16, true);
    constexpr uint64_t kTile = kTileBytes >> 4;  // in a descriptor's units
    const bool lane0 = (threadIdx.x & 31) == 0;
    const uint32_t s_tmem = uniform(sh.tmem) + t * 128, o_tmem = s_tmem + kTmemO;
    const uint32_t base = uniform(smem_u32(sm));
    const uint64_t qd = make_desc_sw128(base, 16) + t * kTile;
    const uint64_t k_major = make_desc_sw128(base, 16) + 2 * kTile;
    const uint64_t mn_major = make_desc_sw128(base, kTileBytes / 2) + 2 * kTile;
    int stage = 0, ring = 0;
    uint32_t phase = 0, ring_phase = 0, q_phase = 0, p_phase = 0, o_phase = 0, turn_phase = t ^ 1;
    for (;;) {
        if (!wait_warp(sh, &sh.item_full[ring], ring_phase)) return;
        const Item it = sh.item[ring];
        __syncwarp();
        if (lane0) mbar_arrive(&sh.item_empty[ring]);
        if (++ring == kRing) ring = 0, ring_phase ^= 1;
        if (uniform(it.head) < 0) return;
        const Tile x = tile_of(a, it, 0), y = tile_of(a, it, 1);
        const Blocks b = blocks_of(x, y);
        const int b_lo = uniform(b.lo), b_hi = uniform(b.hi);
        const int lo = uniform(t ? y.lo : x.lo), hi = uniform(t ? y.hi : x.hi);
        if (b_hi <= b_lo) continue;
        // S of block j; the stage is filled and it is this tile's turn
        auto qk = [&](int j) {
            const bool active = j >= lo && j < hi;
            tc_fence_after();
            const uint64_t kd = k_major + stage * kTile;
            if (active) {
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint64_t off = (s >> 2) * (kTile / 2) + (s & 3) * 2;
                        mma_f16(s_tmem, qd + off, kd + off, kQK, s > 0);
                    }
                    mma_commit(&sh.s_full[t]);
                    mma_commit(&sh.kv_empty[stage]);
                    if (j == hi - 1) mma_commit(&sh.q_empty[t]);
                }
            } else if (lane0) {
                mbar_arrive(&sh.kv_empty[stage]);
            }
            __syncwarp();
            if (++stage == kStages) stage = 0, phase ^= 1;
        };
        auto my_turn = [&] {
            if (!wait_warp(sh, &sh.turn[t], turn_phase)) return false;
            turn_phase ^= 1;
            return true;
        };
        auto pass_turn = [&] {
            __syncwarp();
            if (lane0) mbar_arrive(&sh.turn[t ^ 1]);
        };
        if (!wait_warp(sh, &sh.kv_full[stage], phase)) return;
        if (b_lo == lo && lo < hi) {
            if (!wait_warp(sh, &sh.q_full[t], q_phase)) return;
            q_phase ^= 1;
        }
        if (!my_turn()) return;
        qk(b_lo);
        pass_turn();
        for (int j = b_lo; j < b_hi; ++j) {
            const bool active = j >= lo && j < hi, more = j + 1 < b_hi;
            // everything to wait for comes before the turn
            if (!wait_warp(sh, &sh.kv_full[stage], phase)) return;
            const int v_stage = stage;
            if (++stage == kStages) stage = 0, phase ^= 1;
            if (more && !wait_warp(sh, &sh.kv_full[stage], phase)) return;
            if (more && j + 1 == lo && lo < hi) {
                if (!wait_warp(sh, &sh.q_full[t], q_phase)) return;
                q_phase ^= 1;
            }
            if (active) {
                if (j == lo) {
                    if (!wait_warp(sh, &sh.o_empty[t], o_phase ^ 1)) return;
                    o_phase ^= 1;
                }
                if (!wait_warp(sh, &sh.p_full[t][0], p_phase)) return;
            }
            if (!my_turn()) return;
            if (active) {
                const uint64_t vd = mn_major + v_stage * kTile;
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if (part && !wait_warp(sh, &sh.p_full[t][part], p_phase)) return;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int s = 4 * part + i;
                            mma_f16_ta(o_tmem, s_tmem + 8 * s, vd + s * 128, kPV,
                                       j > lo || part || i);
                        }
                        if (part == 1) {
                            mma_commit(&sh.kv_empty[v_stage]);
                            if (j == hi - 1) mma_commit(&sh.o_full[t]);
                        }
                    }
                    __syncwarp();
                }
                p_phase ^= 1;
            } else if (lane0) {
                mbar_arrive(&sh.kv_empty[v_stage]);
            }
            if (more) qk(j + 1);
            pass_turn();
        }
    }
}

// 2^x, numbers below 2^-126 included: a sum may be close to 2^128, and what brings
// it to 1 is one of them (ex2_approx gives 0 there).
__device__ __forceinline__ float ex2_small(float x) {
    const float h = ex2_approx(0.5f * x);
    return h * h;
}

// Four warps, a thread a row of tile t.  Weights are 2^(c s + shift), c = scale
// log2 e, and their sum l; the row's shift makes the largest weight of the first
// block that the row sees 1 (2^kLift for FP16).
//
// BF16 weights have FP32's range, so a later block may exceed that: the shift
// moves, and l and O with it, once l has passed 2^24, and no block but the
// first needs its maximum (a pass over the block, and the wait for it before the
// first weight).  A row whose scores rise so far within one block that l or O
// leaves that range (2^128) comes out infinite and is done again (attend_row).
// FP16 weights end at 65504: each block's maximum is compared with the shift
// before, and the shift moves where a weight would pass 2^(kLift + 8); blocks
// that are seen whole have their maximum from the load itself (8192 tokens: 386
// us with 64 comparisons a block, 357; without any maximum 337, at that step).  kLift
// keeps weights down to 2^-31 of the largest above FP16's smallest number.
template <bool F16, bool CUT>
__device__ __forceinline__ void softmax_role(const PrefillArgs& a, Shared& sh, int t) {
    const int r = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t row_addr = sh.tmem + ((uint32_t)(r & ~31) << 16);
    const uint32_t s_addr = row_addr + t * 128, o_addr = row_addr + kTmemO + t * 128;
    const int token = r / a.group;
    // of the warp's first and last rows
    const int token_0 = uniform(token), token_1 = __shfl_sync(0xffffffffu, token, 31);
    const float c = a.scale * kLog2e;
    uint32_t s_phase = 0, o_phase = 0, ring_phase = 0;
    int ring = 0;
    for (;;) {
        if (!wait_warp(sh, &sh.item_full[ring], ring_phase)) return;
        const Item it = sh.item[ring];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.item_empty[ring]);
        if (++ring == kRing) ring = 0, ring_phase ^= 1;
        if (it.head < 0) return;
        const Tile tile = tile_of(a, it, t);
        if (tile.hi <= tile.lo) continue;
        // The warp's rows see none of the keys before any_lo and from any_hi on, and
        // all of [all_lo, all_hi): most groups of 32 keys are seen by all of its few
        // tokens or by none, in the first and last blocks too.
        const int pos_0 = tile.pos + token_0, pos_1 = tile.pos + min(token_1, tile.tokens - 1);
        const int any_hi = pos_1 >= pos_0 ? pos_1 + 1 : 0, all_hi = pos_0 + 1;
        const int any_lo = first_seen(pos_0, a.window);
        const int all_lo = first_seen(pos_1, a.window);
        // keys first..pos; a row that is none of the tile's sees none
        const int pos = token < tile.tokens ? tile.pos + token : -1;
        const int first = first_seen(pos, a.window);
        // blocks [clear_lo, clear_hi) are seen whole by all of the tile's rows
        const int clear_hi = (tile.pos + 1) >> 7;
        const int clear_lo =
            a.window ? (max(0, tile.pos + tile.tokens - a.window) + 127) >> 7 : 0;
        float shift = 0.f, l = 0.f;
        for (int j = tile.lo; j < tile.hi; ++j) {
            if (!wait_warp(sh, &sh.s_full[t], s_phase)) return;
            s_phase ^= 1;
            tc_fence_after();
            const bool edge = j < clear_lo || j >= clear_hi;
            // scores of keys 32 i .. 32 i + 31 that the row does not see become -inf
            auto unseen = [&](int i) {
                const int at = j * 128 + 32 * i;
                return at >= any_hi || at + 32 <= any_lo;
            };
            auto hide = [&](float (&x)[32], int i) {
                const int at = j * 128 + 32 * i;
                if (at >= all_lo && at + 32 <= all_hi) return;
                const int from = max(0, min(32, first - j * 128 - 32 * i));
                const int n = max(0, min(32, pos - j * 128 - 32 * i + 1));
                const uint32_t see = (uint32_t)(((1ull << n) - 1) >> from << from);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (!(see >> k & 1)) x[k] = -INFINITY;
            };
            // The shift moves by `by`.  All MMAs before S of this block are done,
            // the last O += P V among them.
            auto move = [&](float by) {
                const float f = ex2_small(by);
                shift += by;
                l *= f;
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    float o[16];
                    uint32_t u[16];
                    tmem_ld16(o_addr + 16 * i, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 16; ++x) u[x] = __float_as_uint(o[x] * f);
                    tmem_st16u(o_addr + 16 * i, u);
                }
            };
            // rows that had not seen a key before this block, and may now
            const bool fresh = l == 0.f && pos >= max(first, j * 128);
            if (F16 || __any_sync(0xffffffffu, fresh)) {
                float top = -INFINITY;
                if (!edge) {
#pragma unroll 1
                    for (int i = 0; i < 128; i += 64) {
                        const float most = tmem_max32(s_addr + i);
                        const float other = tmem_max32(s_addr + i + 32);
                        tmem_ld_wait();
                        top = fmaxf(top, fmaxf(most, other));
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        if (unseen(i)) continue;
                        float x[32], mx[4];
                        tmem_ld32(s_addr + 32 * i, x);
                        tmem_ld_wait();
                        hide(x, i);
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(x[k], x[k + 4]);
#pragma unroll
                        for (int k = 8; k < 32; k += 8)
#pragma unroll
                            for (int n = 0; n < 4; ++n)
                                mx[n] = fmaxf(fmaxf(mx[n], x[k + n]), x[k + n + 4]);
                        top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                        // BF16: any score will do
                        if (!F16 && !__any_sync(0xffffffffu, fresh && top == -INFINITY)) break;
                    }
                }
                if (fresh) shift = (top == -INFINITY ? 0.f : -top * c) + kLift<F16>;
                if (F16) {
                    // Only for rows of the tile that have weights: nothing has waited
                    // for O in an item's first block (the writers may be reading the
                    // last item's), and a row that is none of the tile's, which holds
                    // another sequence's queries, may have any maximum.
                    const float over = fmaf(top, c, shift) - kLift<F16>;
                    const float by = over > 8.f && pos >= 0 && l > 0.f ? -over : 0.f;
                    if (__any_sync(0xffffffffu, by != 0.f)) move(by);
                }
            }
            if (!F16) {
                const bool big = l > kLag && l < INFINITY;  // an infinite sum stays one
                if (__any_sync(0xffffffffu, big)) move(big ? -log2f(l) : 0.f);
            }
            const float2 c2 = make_float2(c, c), b2 = make_float2(shift, shift);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            // 32 keys to weights, written over scores that are no longer needed
            auto weights = [&](const float (&x)[32], int i) {
                uint32_t p[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float2 e = fma2(make_float2(x[2 * k], x[2 * k + 1]), c2, b2);
                    e.x = ex2_approx(e.x);
                    e.y = ex2_approx(e.y);
                    sum[k & 1] = add2(sum[k & 1], e);
                    p[k] = F16 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
                }
                tmem_st16u(s_addr + 16 * i, p);
            };
            // P goes to the MMA warp in two parts (in one: 1504 TFLOP/s at 8192 tokens
            // where two gave 1590).
            auto hand_over = [&](int part) {
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[t][part]);
            };
            // Rolled: two warps of a scheduler are at different places of this code,
            // and what a block takes has to stay in the instruction cache nearest to
            // it (128 keys unrolled: 1354 TFLOP/s at 8192 tokens, 32: 1590; 16: a
            // tenth less again).  For FP16, whose maxima come before, 64 a step with
            // both loads in flight (8192 tokens: 340 us, with 32 352; BF16 323, 321).
            if (!edge) {
                constexpr int kLoads = F16 ? 2 : 1;
#pragma unroll 1
                for (int i = 0; i < 4; i += kLoads) {
                    float x[kLoads][32];
#pragma unroll
                    for (int n = 0; n < kLoads; ++n) tmem_ld32(s_addr + 32 * (i + n), x[n]);
                    tmem_ld_wait();
#pragma unroll
                    for (int n = 0; n < kLoads; ++n) weights(x[n], i + n);
                    if (F16 || (i & 1)) hand_over(i >> 1);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    if (unseen(i)) {
                        const uint32_t zero[16] = {};
                        tmem_st16u(s_addr + 16 * i, zero);
                    } else {
                        float x[32];
                        tmem_ld32(s_addr + 32 * i, x);
                        tmem_ld_wait();
                        hide(x, i);
                        weights(x, i);
                    }
                    if (i & 1) hand_over(i >> 1);
                }
            }
            const float2 both = add2(sum[0], sum[1]);
            l += both.x + both.y;
        }
        // once the writers have read the last item's
        if (!wait_warp(sh, &sh.o_empty[t], o_phase ^ 1)) return;
        o_phase ^= 1;
        sh.sum[t][r] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sum_full[t]);
        if (CUT && it.index < 0)
            a.part_stat[(-1 - it.index) * 256LL + t * 128 + r] = make_float2(shift, l);
        else if (a.lse && token < tile.tokens) {
            const long long row = (long long)it.e.row + t * a.tile_tokens + token;
            a.lse[row * a.heads + it.head * a.group + r - token * a.group] =
                l == 0.f ? -INFINITY : (log2f(l) - shift) * kLn2;
        }
    }
}

// 32 bytes, a whole sector where the address allows.
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

// Four warps that divide by the sum and write finished tiles.
template <bool F16, bool CUT>
__device__ __forceinline__ void write_role(const PrefillArgs& a, Shared& sh) {
    const int r = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t row_addr = sh.tmem + ((uint32_t)(r & ~31) << 16) + kTmemO;
    const int token = r / a.group, in_group = r - token * a.group;
    uint32_t phase[2] = {0, 0}, ring_phase = 0;
    int ring = 0;
    for (;;) {
        if (!wait_warp(sh, &sh.item_full[ring], ring_phase)) return;
        const Item it = sh.item[ring];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.item_empty[ring]);
        if (++ring == kRing) ring = 0, ring_phase ^= 1;
        if (it.head < 0) return;
        const int h = it.head * a.group + in_group;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            const Tile tile = tile_of(a, it, t);
            if (tile.tokens == 0) continue;
            const bool mine = token < tile.tokens;
            const long long row = (long long)it.e.row + t * a.tile_tokens + token;
            uint16_t* dst = a.o + row * a.o_stride + h * D;
            const bool any = tile.hi > tile.lo;
            float l = 0.f;
            if (any) {
                if (!wait_warp(sh, &sh.sum_full[t], phase[t])) return;
                l = sh.sum[t][r];
                if (!wait_warp(sh, &sh.o_full[t], phase[t])) return;
                phase[t] ^= 1;
                tc_fence_after();
            }
            const bool empty = l == 0.f;
            const float inv = empty ? 0.f : 1.f / l;
            float poison = 0.f;  // NaN once any value is not finite
            float* const part =
                CUT && it.index < 0 ? a.part + ((-1 - it.index) * 256LL + t * 128 + r) * D
                                    : nullptr;
            if (part && !any) {
                a.part_stat[(-1 - it.index) * 256LL + t * 128 + r] = make_float2(0.f, 0.f);
                continue;
            }
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                float o[16];
                if (any) {
                    tmem_ld16(row_addr + t * 128 + 16 * i, o);
                    tmem_ld_wait();
                }
                if (part) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        reinterpret_cast<float4*>(part + 16 * i)[x] =
                            make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                    continue;
                }
                uint32_t u[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float y0 = empty ? 0.f : o[2 * x] * inv;
                    const float y1 = empty ? 0.f : o[2 * x + 1] * inv;
                    poison = fmaf(y0, 0.f, poison);
                    poison = fmaf(y1, 0.f, poison);
                    u[x] = narrow2<F16>(y0, y1);
                }
                if (mine) store_32(dst + 16 * i, u);
            }
            if (any) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.o_empty[t]);
            }
            if (part) continue;
            if (!any && mine && a.lse) a.lse[row * a.heads + h] = -INFINITY;
            // a sum that is NaN comes from a key that the row sees
            const unsigned again = __ballot_sync(
                0xffffffffu, mine && ((poison != poison && l == l) || l == INFINITY));
            if (again && lane == 0) {
                const int at = (it.index * 2 + t) * 4 + (r >> 5);
                a.redo[at] = {it.e, it.head, again, atomicExch(&sh.redo, at)};
            }
        }
    }
}

// CUT: items may be shared (a kernel of its own: what that adds slows others down).
// The order of the roles below is that of their code; with the softmax before the
// TMA warp the same prompts took 2 % longer.
template <bool F16, bool CUT>
__global__ void __launch_bounds__(kThreads, 1)
attn_prefill_kernel(PrefillArgs a, const __grid_constant__ CUtensorMap mq,
                    const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv) {
    extern __shared__ __align__(1024) unsigned char sm[];
    Shared& sh = *reinterpret_cast<Shared*>(sm + kSharedOff);
    const int warp = threadIdx.x >> 5;
    if (smem_u32(sm) & 1023u) {  // the swizzle goes by address bits
        if (threadIdx.x == 0) atomicOr(&g_attn_status, STATUS_SMEM_ALIGN);
        return;
    }
    if (threadIdx.x == 0) {
        sh.stop = 0;
        sh.redo = -1;
        for (int i = 0; i < kStages; ++i) mbar_init(&sh.kv_full[i], 1), mbar_init(&sh.kv_empty[i], 2);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh.q_full[t], 1);
            mbar_init(&sh.q_empty[t], 1);
            mbar_init(&sh.s_full[t], 1);
            mbar_init(&sh.turn[t], 1);
            for (int i = 0; i < 2; ++i) mbar_init(&sh.p_full[t][i], 4);
            mbar_init(&sh.o_full[t], 1);
            mbar_init(&sh.o_empty[t], 4);
            mbar_init(&sh.sum_full[t], 4);
        }
        for (int i = 0; i < kRing; ++i) mbar_init(&sh.item_full[i], 1), mbar_init(&sh.item_empty[i], 14);
        fence_mbar_init();
        prefetch_tmap(&mq);
        prefetch_tmap(&mk);
        prefetch_tmap(&mv);
    }
    if (warp == 12) tmem_alloc(&sh.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    if (warp == 14) {
        load_role<CUT>(a, sh, sm, &mq, &mk, &mv);
    } else if (warp < 8) {
        softmax_role<F16, CUT>(a, sh, warp >> 2);
    } else if (warp < 12) {
        write_role<F16, CUT>(a, sh);
    } else {
        if (warp == 12) {
            mma_role<F16, 0>(a, sh, sm);
        } else if (warp == 13) {
            mma_role<F16, 1>(a, sh, sm);
        } else if (!a.list && a.cu_q && blockIdx.x == 0) {
            // with a list, attn_plan_kernel looks at the offsets
            const bool ok = warp_offsets_ok(a.cu_q, a.n_seqs, a.t_q) &&
                            warp_offsets_ok(a.cu_k, a.n_seqs, a.t_k);
            if (!ok && (threadIdx.x & 31) == 0) atomicOr(&g_attn_status, STATUS_BAD_CU_SEQLENS);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(sh.tmem, 512);
    // rows that a masked key's infinity or NaN has reached
    if (warp < 8) {
        for (int at = sh.redo; at >= 0;) {
            const Redo d = a.redo[at];
            const int t = at >> 2 & 1;
            for (int i = warp; i < 32; i += 8) {
                if (!(d.rows >> i & 1)) continue;
                const int r = (at & 3) * 32 + i, token = r / a.group;
                attend_row<F16>(a, (long long)d.e.row + t * a.tile_tokens + token, d.e.k0,
                                d.e.pos + t * a.tile_tokens + token,
                                d.head * a.group + r - token * a.group);
            }
            at = d.before;
        }
    }
}

// Joins the parts of a call whose items are shared by several CTAs: a row to a
// warp, four channels a lane.
constexpr int kJoinWarps = 8;
template <bool F16>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_prefill_join_kernel(PrefillArgs a) {
    const int lane = threadIdx.x & 31;
    const long long at = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    pdl_wait();
    Item it;
    const int index = (int)(at >> 8), t = (int)(at >> 7) & 1, r = (int)at & 127;
    it.from = 0;
    it.to = 0x7fffffff;
    if (a.list || a.one) {
        if (a.shared + index >= entry_count(a) * a.kv_heads) return;
        ordered_item(a, a.shared + index, it);
    } else {
        const int slot = index / a.kv_heads;
        const int n = warp_find_last(a.n_seqs, slot, [&](int i) { return first_slot(a, i); });
        if (!slot_entry(a, n, slot, it.e)) return;
        it.head = index - slot * a.kv_heads;
    }
    const Tile tile = tile_of(a, it, t);
    const int token = r / a.group;
    if (token >= tile.tokens) return;
    const long long first = ((long long)index * a.splits << 8) + t * 128 + r;
    // up to 152 parts: their factors a lane each, then their channels
    float least = INFINITY, sum = 0.f;
    for (int p = lane; p < a.splits; p += 32) {
        const float2 s = __ldcg(a.part_stat + first + 256LL * p);
        if (s.y != 0.f) least = fminf(least, s.x);
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
        least = fminf(least, __shfl_xor_sync(0xffffffffu, least, off));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < a.splits; p0 += 32) {
        float f = 0.f;
        if (p0 + lane < a.splits) {
            const float2 s = __ldcg(a.part_stat + first + 256LL * (p0 + lane));
            if (s.y != 0.f) {
                f = ex2_small(least - s.x);
                // (an infinite sum stays one, however small its factor)
                sum = s.y < INFINITY ? fmaf(s.y, f, sum) : sum + s.y;
            }
        }
        const int here = min(32, a.splits - p0);
#pragma unroll 4
        for (int i = 0; i < here; ++i) {
            const float fi = __shfl_sync(0xffffffffu, f, i);
            if (fi == 0.f) continue;  // (nothing was written where there was no key)
            const float4 x = __ldcg(
                reinterpret_cast<const float4*>(a.part + (first + 256LL * (p0 + i)) * D) + lane);
            o.x = fmaf(x.x, fi, o.x);
            o.y = fmaf(x.y, fi, o.y);
            o.z = fmaf(x.z, fi, o.z);
            o.w = fmaf(x.w, fi, o.w);
        }
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const int h = it.head * a.group + r - token * a.group;
    const long long row = (long long)it.e.row + t * a.tile_tokens + token;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    const float poison = (o.x + o.y + o.z + o.w) * 0.f;
    if (__any_sync(0xffffffffu, (poison != poison && sum == sum) || sum == INFINITY)) {
        attend_row<F16>(a, row, it.e.k0, tile.pos + token, h);
        return;
    }
    *reinterpret_cast<uint2*>(a.o + row * a.o_stride + h * D + 4 * lane) =
        make_uint2(narrow2<F16>(o.x, o.y), narrow2<F16>(o.z, o.w));
    if (a.lse && lane == 0)
        a.lse[row * a.heads + h] =
            sum == 0.f ? -INFINITY : (log2f(sum) - least) * kLn2;
}

// Items of a call, at most: slots of all sequences.
inline long long slot_count(long long rows, int n_seqs, int group) {
    return rows / (2 * (128 / group)) + n_seqs;
}
// CTAs that may share an item's keys where items are few, on kSms
// multiprocessors or more: the workspace is sized for so many.
constexpr int kSms = 152;
inline int most_splits(long long items) { return items * 2 <= kSms ? (int)(kSms / items) : 1; }
constexpr size_t kPartBytes = 256 * (128 + 2) * sizeof(float);
// Items of about one length that are more than kSms, but no large multiple of it:
// those of the last round are cut into shares, so that it ends about everywhere at
// once.  How many shares, or 1 where that gains little; more cost more to join.
inline int last_round_splits(long long items, long long& shared) {
    shared = items / kSms * kSms;
    const long long rest = items - shared;
    int best = 1;
    double least = 1. - 0.02 * (double)(items / kSms);
    for (int s = 2; s <= 6 && rest; ++s) {
        const double rounds = (double)((rest * s + kSms - 1) / kSms) / s + 0.01 * s;
        if (items > kSms && rounds < least) least = rounds, best = s;
    }
    return best;
}
// Items of the one sequence there is.
inline long long one_sequence_items(long long rows, int group, int kv_heads) {
    const int tokens = 2 * (128 / group);
    return (rows + tokens - 1) / tokens * kv_heads;
}

}  // namespace

cudaError_t status_word_attn(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_attn_status);
}

kda_status validate_rows(const char* fn, const char* name, const void* p, int64_t stride,
                         int heads) {
    KDA_REQUIRE(p, KDA_ERR_INVALID_ARG, "%s: null pointer argument (%s)", fn, name);
    KDA_REQUIRE(aligned16(p), KDA_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", fn, name);
    KDA_REQUIRE(stride >= (int64_t)heads * D && stride % 8 == 0, KDA_ERR_INVALID_ARG,
                "%s: %s row stride %lld must be >= heads * 128 and a multiple of 8 elements", fn,
                name, (long long)stride);
    return KDA_OK;
}

}  // namespace kda

using namespace kda;

extern "C" size_t kda_attn_prefill_workspace_size(int64_t rows, int n_seqs, int heads,
                                                  int kv_heads) {
    if (rows < 0 || n_seqs < 1 || heads < 1 || kv_heads < 1 || heads % kv_heads ||
        heads / kv_heads > 128)
        return 0;
    // the ticket counter, 32 bytes an entry, 4 a sequence, eight records of rows
    // to be done again per item
    const size_t slots = (size_t)slot_count(rows, n_seqs, heads / kv_heads);
    const size_t items = slots * kv_heads;
    size_t parts = most_splits((long long)items) > 1 ? most_splits((long long)items) * items : 0;
    if (n_seqs == 1) {
        const long long exact = one_sequence_items(rows, heads / kv_heads, kv_heads);
        long long shared;
        const int splits = last_round_splits(exact, shared);
        if (splits > 1) parts = std::max(parts, (size_t)(exact - shared) * splits);
    }
    return 256 + 32 * slots + 16 * (((size_t)n_seqs + 3) / 4) + 8 * sizeof(Redo) * items +
           parts * kPartBytes;
}

extern "C" kda_status kda_attn_prefill(const void* q, const void* k, const void* v, void* o,
                                       float* lse, int t_q, int t_k, const int* cu_seqlens_q,
                                       const int* cu_seqlens_k, int n_seqs, int heads,
                                       int kv_heads, int head_dim, int in_dtype,
                                       int64_t q_row_stride, int64_t k_row_stride,
                                       int64_t v_row_stride, int64_t o_row_stride, int window,
                                       float scale, void* workspace, size_t workspace_bytes,
                                       uint64_t stream) {
    const char* fn = "kda_attn_prefill";
    KDA_REQUIRE(head_dim == D, KDA_ERR_UNSUPPORTED, "%s: head_dim %d unsupported (only 128)", fn,
                head_dim);
    KDA_REQUIRE(in_dtype == KDA_F32 || in_dtype == KDA_BF16 || in_dtype == KDA_F16,
                KDA_ERR_INVALID_ARG, "%s: in_dtype %d is not a kda_dtype", fn, in_dtype);
    KDA_REQUIRE(in_dtype != KDA_F32, KDA_ERR_UNSUPPORTED, "%s: FP32 inputs are not built", fn);
    KDA_REQUIRE(n_seqs >= 1 && t_q >= 0 && t_k >= 0, KDA_ERR_INVALID_ARG,
                "%s: n_seqs (%d) must be >= 1, t_q (%d) and t_k (%d) >= 0", fn, n_seqs, t_q, t_k);
    KDA_REQUIRE(heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0, KDA_ERR_INVALID_ARG,
                "%s: heads (%d) must be a positive multiple of kv_heads (%d)", fn, heads,
                kv_heads);
    KDA_REQUIRE(heads / kv_heads <= 128, KDA_ERR_UNSUPPORTED,
                "%s: %d query heads per KV head (at most 128)", fn, heads / kv_heads);
    KDA_REQUIRE(window >= 0, KDA_ERR_INVALID_ARG, "%s: window (%d) must be >= 0", fn, window);
    KDA_REQUIRE(std::isfinite(scale) && scale > 0.f, KDA_ERR_INVALID_ARG,
                "%s: scale must be finite and positive", fn);
    KDA_REQUIRE(!cu_seqlens_q == !cu_seqlens_k, KDA_ERR_INVALID_ARG,
                "%s: cu_seqlens_q and cu_seqlens_k come together", fn);
    const long long rows_q = cu_seqlens_q ? t_q : (long long)t_q * n_seqs;
    const long long rows_k = cu_seqlens_q ? t_k : (long long)t_k * n_seqs;
    KDA_REQUIRE(rows_q < 0x7fffffffLL && rows_k < 0x7fffffffLL, KDA_ERR_INVALID_ARG,
                "%s: more than 2^31 - 2 token rows", fn);
    if (rows_q == 0) return KDA_OK;
    kda_status st = validate_rows(fn, "q", q, q_row_stride, heads);
    if (st == KDA_OK) st = validate_rows(fn, "o", o, o_row_stride, heads);
    if (st == KDA_OK && rows_k) st = validate_rows(fn, "k", k, k_row_stride, kv_heads);
    if (st == KDA_OK && rows_k) st = validate_rows(fn, "v", v, v_row_stride, kv_heads);
    if (st != KDA_OK) return st;
    const int group = heads / kv_heads, tokens = 128 / group;
    const long long slots = slot_count(rows_q, n_seqs, group);
    KDA_REQUIRE(slots < 0x0fffffffLL / kv_heads, KDA_ERR_INVALID_ARG, "%s: problem too large", fn);
    const size_t need = kda_attn_prefill_workspace_size(rows_q, n_seqs, heads, kv_heads);
    KDA_REQUIRE(workspace && workspace_bytes >= need, KDA_ERR_WORKSPACE,
                "%s: workspace of %zu B, %zu B needed", fn, workspace ? workspace_bytes : 0, need);
    KDA_REQUIRE(aligned16(workspace), KDA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned",
                fn);
    KDA_REQUIRE(!fault_injected(), KDA_ERR_CUDA, "%s: injected launch failure", fn);
    const int sms = sm_count();
    KDA_REQUIRE(sms > 0, KDA_ERR_CUDA, "%s: no device", fn);
    const bool f16 = in_dtype == KDA_F16;
    // without keys nothing is loaded through the K and V maps
    const void* kb = rows_k ? k : q;
    const void* vb = rows_k ? v : q;
    const uint64_t k_rows = rows_k ? (uint64_t)rows_k : 1;
    CUtensorMap mq, mk, mv;
    KDA_REQUIRE(
        tma_map_heads(&mq, q, heads, rows_q, q_row_stride, group, tokens, f16) &&
            tma_map_heads(&mk, kb, rows_k ? kv_heads : heads, k_rows,
                          rows_k ? k_row_stride : q_row_stride, 1, 128, f16) &&
            tma_map_heads(&mv, vb, rows_k ? kv_heads : heads, k_rows,
                          rows_k ? v_row_stride : q_row_stride, 1, 128, f16),
        KDA_ERR_CUDA, "%s: cannot describe the inputs to the copy engine", fn);
    // One CTA per item needs no order and no tickets: the call is one kernel.
    const long long items = slots * kv_heads;
    const bool direct = items <= sms;
    // Few items behind many keys: CTAs share an item's keys, at least four blocks
    // to each, and a second kernel joins them (16 tokens behind 30000, 32 heads
    // over 8: 39 us where one CTA an item takes 304).
    const int blocks = (t_k + 127) / 128;
    int splits = direct ? std::min(most_splits(items), blocks / 4) : 1;
    if (splits < 1 || sms < kSms) splits = 1;
    // A chunk behind a long context: the last round's likewise (32 heads over 8, 2048
    // tokens behind 30000: 672 us without, 630; 1536: 657, 487; 8192: 2710, 2700).
    // Against shorter contexts shares' sums weigh more (all keys without, with
    // shares: 2048 tokens, 8192 keys: 160 us, 182; 12288: 247, 258; 20480: 434, 411;
    // 2500, 10000: 279, 280; 15000: 446, 356; 4096, 16384: 633, 582; under four times
    // the tokens: 4096, 12288: 434, 417, 2048 and less the same).
    long long shared = 0, joins = splits > 1 ? items : 0;
    if (!direct && n_seqs == 1 && t_k >= 4LL * t_q) {
        const long long exact = one_sequence_items(rows_q, group, kv_heads);
        splits = last_round_splits(exact, shared);
        const int seen = window ? std::min(t_k, window) : t_k;
        if (sms < kSms || seen / 128 < 16 * splits) splits = 1;
        if (splits > 1) joins = exact - shared;
    }
    // One sequence's items need no plan, and in a few rounds there and back no
    // counter; in more the counter's evenness is worth more than the plan's time
    // (4096 tokens, 32 heads over 8: 94.1 us with both, 91.3 without; 8192: 322,
    // 321; 32768: 4731, 4850).
    const bool one = !direct && n_seqs == 1 && splits == 1 && items <= 4LL * sms;
    int shift = 0;  // buckets of 2^shift key blocks in the plan's sort
    while ((t_k / 128 >> shift) >= kPlanThreads) ++shift;
    unsigned* count = static_cast<unsigned*>(workspace);
    int4* list = reinterpret_cast<int4*>(static_cast<unsigned char*>(workspace) + 256);
    int4* group_of = list + slots;
    int* first_entry = reinterpret_cast<int*>(group_of + slots);
    Redo* redo = reinterpret_cast<Redo*>(first_entry + 4 * ((n_seqs + 3LL) / 4));
    float* part = reinterpret_cast<float*>(redo + 8 * items);
    float2* part_stat = reinterpret_cast<float2*>(part + 256LL * D * joins * splits);
    PrefillArgs a = {(const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v, (uint16_t*)o,
                     lse, cu_seqlens_q, cu_seqlens_k, q_row_stride, k_row_stride, v_row_stride,
                     o_row_stride, t_q, t_k, n_seqs, heads, kv_heads, window, group, tokens,
                     scale, direct || one ? nullptr : list, one, group_of, first_entry, count,
                     redo, (int)slots, shift, splits, (int)shared, part, part_stat};
    auto kernel = splits > 1 ? attn_prefill_kernel<false, true> : attn_prefill_kernel<false, false>;
    if (f16)
        kernel = splits > 1 ? attn_prefill_kernel<true, true> : attn_prefill_kernel<true, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    if (e != cudaSuccess) {
        set_error("%s: cannot reserve shared memory: %s", fn, cudaGetErrorString(e));
        return KDA_ERR_CUDA;
    }
    cudaStream_t s = as_stream(stream);
    if (!direct && !one) launch_pdl(attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a);
    launch_pdl(kernel, dim3((unsigned)(direct ? items * splits : sms)), dim3(kThreads), kSmemBytes,
               s, a, mq, mk, mv);
    if (splits > 1)
        launch_pdl(f16 ? attn_prefill_join_kernel<true> : attn_prefill_join_kernel<false>,
                   dim3((unsigned)(joins * 256 / kJoinWarps)), dim3(kJoinWarps * 32), 0, s, a);
    return launch_result(fn);
}
