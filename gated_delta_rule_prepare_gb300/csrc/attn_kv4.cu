// The paged 4-bit key/value cache: its writer (kda_attn_kv4_append) and its
// reader (kda_attn_kv4_read).  The decode over it is in attn_decode.cu.
//
// Per token, KV head and 64 channels, with x the row's values:
//     m = the largest BF16 <= min x,  s = the smallest BF16 >= (max x - m) / 15
//     code = round((x - m) / s) to nearest, ties to even, 0 where s = 0
// and a code stands for m + s * code.  All three are functions of the real
// numbers, not of a rounding on the way: the kernel gets them from directed
// FP32 operations and decides values near a border between two codes apart.
//
// Both kernels give one warp 16 tokens of one head: one group of the cache, 1024
// bytes of codes, staged in shared memory so that global memory sees 16-byte
// accesses on both sides; of K and then of V, or with few tokens one of them.
// Memory-bound in principle, 512 + 144 bytes per (token, head); at the front
// end's batch (88 thousand tokens, 8 heads) read takes 67 us, 5.8 TB/s, and
// append 110 us, 4.2 TB/s, bound by the issue of its exact rounding's instructions.
#include "attn_common.h"
#include "f32x2.h"

namespace kda {
namespace {

using namespace attn;

__device__ unsigned g_kv4_status = 0;

constexpr int kWarps = 4;
// The second half of a staged group (channels 64..127) starts 32 bytes late,
// so that lanes of both halves use different banks.
constexpr int kStage = 1024 + 32;
__device__ __forceinline__ int staged(int byte) { return byte + (byte >> 9) * 32; }

struct RowArgs {
    uint16_t *k, *v;
    long long k_stride, v_stride;
    const int* cu;
    int t, n_seqs;
    Cache c;
};

// What a warp works on: `count` rows from packed row `row`, positions from
// `pos`, of sequence `n`; the rows lie in one 16-token group of the cache.
struct Slot {
    int n, pos, count;
    long long row;
};

// Slots are numbered so that a sequence whose rows start at packed row c owns
// slots from c / 16 + 2 n: r rows touch at most (r + 30) / 16 groups, which is
// never more than the distance to the next sequence's first slot.
__device__ __forceinline__ bool find_slot(const RowArgs& a, long long slot, Slot& s) {
    long long row0;
    int rows;
    if (a.cu) {
        s.n = warp_find_last(a.n_seqs, slot,
                             [&](int i) { return (long long)(__ldg(a.cu + i) / 16) + 2LL * i; });
        const int c0 = __ldg(a.cu + s.n), c1 = __ldg(a.cu + s.n + 1);
        if (c0 < 0 || c1 < c0 || c1 > a.t) return false;
        row0 = c0;
        rows = c1 - c0;
    } else {
        s.n = warp_find_last(a.n_seqs, slot,
                             [&](int i) { return (long long)i * a.t / 16 + 2LL * i; });
        row0 = (long long)s.n * a.t;
        rows = a.t;
    }
    const int len = __ldg(a.c.lens + s.n);
    const int first = len - rows;  // position of the sequence's first row
    if (len < 0 || first < 0 || (long long)len > ((long long)a.c.max_pages << a.c.page_shift)) {
        if (rows > 0 && (threadIdx.x & 31) == 0) atomicOr(&g_kv4_status, STATUS_BAD_PAGES);
        return false;
    }
    const long long g = slot - (row0 / 16 + 2LL * s.n);
    const long long from = (long long)(first & ~15) + g * 16;
    if (g < 0 || from >= len) return false;
    s.pos = max(first, (int)from);
    s.count = min(len - (int)from, 16) - (s.pos - (int)from);
    s.row = row0 + (s.pos - first);
    return s.count > 0;
}

__device__ __forceinline__ void check_offsets(const RowArgs& a) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 32 && a.cu &&
        !warp_offsets_ok(a.cu, a.n_seqs, a.t) && threadIdx.x == 0)
        atomicOr(&g_kv4_status, STATUS_BAD_CU_SEQLENS);
}

// Minimum and maximum of two elements at a time, NaN if either is.
template <bool F16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (F16) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (F16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// BF16 bits of x rounded towards minus infinity, and of x >= 0 towards plus
// infinity (x finite).
__device__ __forceinline__ uint32_t bf16_down(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u >> 16) + ((u >> 31) && (u & 0xffffu) ? 1u : 0u);
}
__device__ __forceinline__ uint32_t bf16_up(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u >> 16) + ((u & 0xffffu) ? 1u : 0u);
}

// The code of x by comparison with borders, for groups whose numbers lie too far
// apart for codes8: t + e is x - m exactly (the rounded difference and what it
// lost), and the fused multiply-add gets the sign of t - (c + 0.5) s right.
__device__ __noinline__ uint32_t code_exact(float x, float m, float s) {
    if (s >= 1e37f) x *= 0.25f, m *= 0.25f, s *= 0.25f;  // exact, and x - m finite
    const float t = x - m;
    const float back = x - t;
    const float e = (x - (t + back)) + (back - m);
    float c = fminf(fmaxf(floorf(t / s) - 1.f, -1.f), 15.f);
    for (int i = 0; i < 3 && c < 15.f; ++i) {
        const float d = fmaf(-(c + 0.5f), s, t);
        const bool above = d > 0.f || (d == 0.f && (e > 0.f || (e == 0.f && ((int)c & 1))));
        if (!above) break;
        c += 1.f;
    }
    return (uint32_t)fminf(fmaxf(c, 0.f), 15.f);
}

// Eight channels of one token row: codes packed four bits each, channel x in
// bits 4x.  With k = floor of the quotient (which may be off by one where the
// quotient is close to an integer: that moves nothing) the code is k or k + 1, as
// x lies below or above the border b = m + (k + 0.5) s, and the even one of them
// on it.  k + 0.5 has 5 bits and s has 8, so b is exact in FP32 unless m and s are
// more than 2^10 apart: ten operations a value, no case apart for ties
// (of BF16 rows some 1 in 300 values is one; deciding those in a branch took
// 640 us for the front end's batch where this takes 110).
__device__ __forceinline__ float2 fma2_down(float2 a, float2 b, float2 c) {  // rounded down
    unsigned long long r;
    asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)), "l"(pk(c)));
    return upk(r);
}

template <bool F16>
__device__ __forceinline__ uint32_t codes8(const uint4& raw, float m, float s, float inv) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t out = 0;
    if (inv != 0.f) {  // m and s are near enough
        constexpr float kMagic = 8388608.f;  // 2^23: integers above it are their last bits
        constexpr uint32_t kBits = 0x4b000000u;
        const float2 inv2 = make_float2(inv, inv), s2 = make_float2(s, s), m2 = make_float2(m, m);
        const float2 less_m = make_float2(-m, -m), magic = make_float2(kMagic, kMagic);
        const float2 half = make_float2(0.5f - kMagic, 0.5f - kMagic);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = widen2<F16>(w[i]);
            const float2 k = fma2_down(add2(x, less_m), inv2, magic);
            const float2 b = fma2(add2(k, half), s2, m2);
            const float2 d = add2(b, make_float2(-x.x, -x.y));
            // one more where b - x is negative, or zero and k odd: where its bits,
            // less k's last one, have the sign bit
            const uint32_t k0 = __float_as_uint(k.x), k1 = __float_as_uint(k.y);
            const uint32_t c0 = k0 + ((__float_as_uint(d.x) - (k0 & 1)) >> 31);
            const uint32_t c1 = k1 + ((__float_as_uint(d.y) - (k1 & 1)) >> 31);
            // (as multiply-adds: the shifts and ANDs of this loop bound it)
            asm("mad.lo.u32 %0, %1, %2, %0;" : "+r"(out) : "r"(c0), "r"(1u << (8 * i)));
            asm("mad.lo.u32 %0, %1, %2, %0;" : "+r"(out) : "r"(c1), "r"(1u << (8 * i + 4)));
        }
        return out - (kBits + (kBits << 4));
    }
    if (!(s > 0.f)) return 0u;
    for (int i = 0; i < 4; ++i) {
        const float2 x = widen2<F16>(w[i]);
        out |= code_exact(x.x, m, s) << (8 * i) | code_exact(x.y, m, s) << (8 * i + 4);
    }
    return out;
}

// 16 tokens of one head of K or of V, by one warp.
template <bool F16>
__device__ __forceinline__ void append_group(const RowArgs& a, const Slot& s, uint8_t* stage,
                                             uint8_t* block, int h, bool is_v) {
    const int lane = threadIdx.x & 31;
    const long long stride = is_v ? a.v_stride : a.k_stride;
    const uint16_t* src = (is_v ? a.v : a.k) + h * D;
    const int hw = lane >> 4, c = lane & 15, b = c >> 1;
    const int t0 = s.pos & 15;  // first token of the group that is written
    uint4 raw[8];
    src += (s.row - t0 + hw) * stride + 8 * c;
    if (s.count == 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            raw[j] = __ldg(reinterpret_cast<const uint4*>(src + 2 * j * stride));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int tok = 2 * j + hw;
            raw[j] = tok >= t0 && tok < t0 + s.count
                         ? __ldg(reinterpret_cast<const uint4*>(src + 2 * j * stride))
                         : make_uint4(0, 0, 0, 0);
        }
    }
    const int in_page = s.pos & (a.c.page() - 1) & ~15;
    uint8_t* par = block + a.c.page() * 64 + (long long)in_page * 8;
    // Least and greatest of each token's 64 channels, over eight lanes, so that
    // lane c % 8 = j ends with token j's: 4 + 2 + 1 exchanges for 8 tokens.
    uint32_t mm[8];  // (least, greatest) of this lane's channels, both 16 bits
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t lo = min2<F16>(min2<F16>(raw[j].x, raw[j].y), min2<F16>(raw[j].z, raw[j].w));
        const uint32_t hi = max2<F16>(max2<F16>(raw[j].x, raw[j].y), max2<F16>(raw[j].z, raw[j].w));
        // (lo.x, -hi.x) and (lo.y, -hi.y): one minimum serves both
        constexpr uint32_t kMinus = 0x80000000u;
        mm[j] = min2<F16>(__byte_perm(lo, hi, 0x5410) ^ kMinus, __byte_perm(lo, hi, 0x7632) ^ kMinus);
    }
#pragma unroll
    for (int half = 4; half >= 1; half /= 2) {
        const bool up = c & half;
#pragma unroll
        for (int j = 0; j < half; ++j) {
            const uint32_t give = up ? mm[j] : mm[j + half];
            const uint32_t keep = up ? mm[j + half] : mm[j];
            mm[j] = min2<F16>(keep, __shfl_xor_sync(0xffffffffu, give, half));
        }
    }
    // token 2 (c % 8) + hw: parameters, and 1 / s, or 0 where m and s lie too far
    // apart for codes8
    float my_m, my_s, my_inv;
    {
        const float2 x = widen2<F16>(mm[0]);
        uint32_t mb = bf16_down(x.x);
        my_m = __uint_as_float(mb << 16);
        // both rounded up: at or above the real quotient, and equal to it where it
        // is a BF16 number (of quarters where the difference may pass FP32's range)
        const bool huge = fmaxf(fabsf(my_m), fabsf(x.y)) > 1e38f;
        const float q = huge ? 4.f * __fdiv_ru(__fsub_ru(-0.25f * x.y, 0.25f * my_m), 15.f)
                             : __fdiv_ru(__fsub_ru(-x.y, my_m), 15.f);
        uint32_t sb = bf16_up(q);
        // an infinity or a NaN in the group: every value of it reads as NaN
        const bool bad = !(q < 3e38f) || !(fabsf(my_m) < INFINITY);
        if (bad) mb = sb = 0x7fffu;
        my_s = bad ? 0.f : __uint_as_float(sb << 16);
        if (bad) my_m = 0.f;
        const float size = fabsf(my_m);
        const bool plain = my_s > 1e-30f && my_s < 1e37f && size <= 1024.f * my_s &&
                           (size == 0.f || my_s <= 1024.f * size);
        my_inv = plain ? 1.f / my_s : 0.f;
        const int tok = 2 * (c & 7) + hw;
        if (tok >= t0 && tok < t0 + s.count)
            *reinterpret_cast<uint32_t*>(par + tok * 8 + (c >> 3) * 4) = sb | mb << 16;
    }
    // Codes of tokens tok and tok + 8 at a time: of K, the four bytes of a word.
    // An even lane holds channels 16 b + x, its odd neighbour 16 b + 8 + x, and
    // they store x = 0..3 and x = 4..7.
    const bool odd = lane & 1;
    __syncwarp();  // the last group's codes have been read
    uint8_t* const dst = stage + staged(512 * (b >> 2)) + 4 * (b & 3);
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
        uint32_t own[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int from = (lane & ~7) | (jj + 4 * n);
            own[n] = codes8<F16>(raw[jj + 4 * n], __shfl_sync(0xffffffffu, my_m, from),
                                 __shfl_sync(0xffffffffu, my_s, from),
                                 __shfl_sync(0xffffffffu, my_inv, from));
        }
        // low halves are x = 0..3; the neighbour gets the half it stores
        const uint32_t low = __byte_perm(own[0], own[1], 0x5410);
        const uint32_t high = __byte_perm(own[0], own[1], 0x7632);
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? low : high, 1);
        const uint32_t nib0 = odd ? got : low, nib1 = odd ? high : got;
        const uint32_t e = (nib0 & 0x0f0f0f0fu) | (nib1 & 0x0f0f0f0fu) << 4;
        const uint32_t o = (nib0 >> 4 & 0x0f0f0f0fu) | (nib1 & 0xf0f0f0f0u);
        const uint32_t w0 = __byte_perm(e, o, 0x6420), w1 = __byte_perm(e, o, 0x7531);
        if (!is_v) {
            // token g = 2 jj + hw: words t = 0..3 at 16 (4 g + t)
            uint32_t* p = reinterpret_cast<uint32_t*>(dst + 64 * (2 * jj + hw) + (odd ? 32 : 0));
            p[0] = w0;
            p[4] = w1;
        } else {
            // t = jj, e = hw: channel x at 16 (4 x + t) + 2 e
            uint8_t* p = dst + 16 * jj + 2 * hw + (odd ? 256 : 0);
            *reinterpret_cast<uint16_t*>(p) = (uint16_t)w0;
            *reinterpret_cast<uint16_t*>(p + 64) = (uint16_t)(w0 >> 16);
            *reinterpret_cast<uint16_t*>(p + 128) = (uint16_t)w1;
            *reinterpret_cast<uint16_t*>(p + 192) = (uint16_t)(w1 >> 16);
        }
    }
    __syncwarp();
    uint8_t* codes = block + (long long)in_page * 64;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int at = half * 512 + lane * 16;
        const uint4 v = *reinterpret_cast<const uint4*>(&stage[staged(at)]);
        if (s.count == 16) {
            *reinterpret_cast<uint4*>(codes + at) = v;
            continue;
        }
        // a byte belongs to one token: the others of the group stay as they are
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int e = i >> 1 & 1, hi8 = i & 1;
            const int tok = 8 * hi8 + (is_v ? 2 * (lane & 3) + e : lane >> 2);
            if (tok >= t0 && tok < t0 + s.count)
                codes[at + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
        }
    }
}

// grid (ceil(slots / 4), kv_heads, 1 or 2): a warp does K and then V of its 16
// tokens, or with two one of them.  A half-warp
// loads a token row of 128 channels, 16 bytes a lane, all sixteen tokens of
// the group in flight.
template <bool F16>
__global__ void __launch_bounds__(kWarps * 32, 8) append_kernel(RowArgs a) {
    __shared__ __align__(16) uint8_t stage[kWarps][kStage];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    check_offsets(a);
    Slot s;
    if (!find_slot(a, (long long)blockIdx.x * kWarps + warp, s)) return;  // whole warps
    const int h = blockIdx.y;
    uint8_t* block = a.c.block(s.n, s.pos, h);
    if (!block) {
        if (lane == 0) atomicOr(&g_kv4_status, STATUS_BAD_PAGES);
        return;
    }
#pragma unroll 1
    for (int which = blockIdx.z; which < 2; which += gridDim.z)
        append_group<F16>(a, s, stage[warp], block + which * part_bytes(a.c.page()), h, which);
}

// The same the other way: a lane turns 8 channels of a token into 16 bytes.
template <bool F16>
__device__ __forceinline__ void read_group(const RowArgs& a, const Slot& s, uint8_t* stage,
                                           const uint8_t* block, int h, bool is_v) {
    const int lane = threadIdx.x & 31;
    const long long stride = is_v ? a.v_stride : a.k_stride;
    const int hw = lane >> 4, c = lane & 15, b = c >> 1;
    const int t0 = s.pos & 15;
    const int in_page = s.pos & (a.c.page() - 1) & ~15;
    uint16_t* dst = (is_v ? a.v : a.k) + h * D + 8 * c + (s.row - t0) * stride;
    const uint8_t* par = nullptr;
    __syncwarp();  // the last group's codes have been read
    if (block) {
        par = block + a.c.page() * 64 + (long long)in_page * 8 + (c >> 3) * 4;
        const uint8_t* codes = block + (long long)in_page * 64;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int at = half * 512 + lane * 16;
            *reinterpret_cast<uint4*>(&stage[staged(at)]) =
                __ldg(reinterpret_cast<const uint4*>(codes + at));
        }
    }
    __syncwarp();
    const uint8_t* mine = stage + staged(512 * (b >> 2)) + 4 * (b & 3);
    const int sh = 4 * (lane & 1);
    // One token: code(x) has the code of its channel x = 0..7 of this lane as the
    // FP32 number 2^23 + code.
    auto put = [&](int tok, auto code) {
        if (tok < t0 || tok >= t0 + s.count) return;
        // a page that is not there reads as NaN
        const uint32_t p = par ? __ldg(reinterpret_cast<const uint32_t*>(par + tok * 8))
                               : 0x7fff7fffu;
        const float sc = __uint_as_float(p << 16), m = __uint_as_float(p & 0xffff0000u);
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[i] = narrow2<F16>(fmaf(sc, code(2 * i) - 8388608.f, m),
                                  fmaf(sc, code(2 * i + 1) - 8388608.f, m));
        *reinterpret_cast<uint4*>(dst + tok * stride) = make_uint4(out[0], out[1], out[2], out[3]);
    };
    auto number = [](uint32_t w, int byte) {
        return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7550 + byte));
    };
    if (!is_v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int g = 2 * j + hw;  // tokens g and g + 8 share words t = 0..3
            uint32_t w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                w[t] = *reinterpret_cast<const uint32_t*>(mine + 16 * (4 * g + t)) >> sh &
                       0x0f0f0f0fu;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                put(g + 8 * i, [&](int x) { return number(w[x >> 1], 2 * (x & 1) + i); });
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = 2 * j + hw;  // tokens 2t, 2t + 1, 2t + 8, 2t + 9 share words x = 0..7
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x)
                w[x] = *reinterpret_cast<const uint32_t*>(mine + 16 * (4 * x + t)) >> sh &
                       0x0f0f0f0fu;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    put(2 * t + e + 8 * i, [&](int x) { return number(w[x], 2 * e + i); });
        }
    }
}

template <bool F16>
__global__ void __launch_bounds__(kWarps * 32, 12) read_kernel(RowArgs a) {
    __shared__ __align__(16) uint8_t stage[kWarps][kStage];
    const int warp = threadIdx.x >> 5;
    check_offsets(a);
    Slot s;
    if (!find_slot(a, (long long)blockIdx.x * kWarps + warp, s)) return;
    const int h = blockIdx.y;
    const uint8_t* block = a.c.block(s.n, s.pos, h);
    if (!block && (threadIdx.x & 31) == 0) atomicOr(&g_kv4_status, STATUS_BAD_PAGES);
#pragma unroll 1
    for (int which = blockIdx.z; which < 2; which += gridDim.z)
        read_group<F16>(a, s, stage[warp],
                        block ? block + which * part_bytes(a.c.page()) : nullptr, h, which);
}

kda_status rows_call(const char* fn, bool append, void* k, void* v, int64_t k_stride,
                     int64_t v_stride, int t, const int* cu, int n_seqs, int kv_heads,
                     int head_dim, int in_dtype, uint8_t* cache, int64_t n_pages, int page,
                     const int* table, int max_pages, const int* lens, uint64_t stream) {
    KDA_REQUIRE(in_dtype == KDA_F32 || in_dtype == KDA_BF16 || in_dtype == KDA_F16,
                KDA_ERR_INVALID_ARG, "%s: in_dtype %d is not a kda_dtype", fn, in_dtype);
    KDA_REQUIRE(in_dtype != KDA_F32, KDA_ERR_UNSUPPORTED, "%s: FP32 rows are not built", fn);
    KDA_REQUIRE(t >= 0, KDA_ERR_INVALID_ARG, "%s: t (%d) must be >= 0", fn, t);
    kda_status st = validate_cache(fn, cache, n_pages, page, table, max_pages, lens, n_seqs,
                                   kv_heads, head_dim);
    if (st != KDA_OK) return st;
    if (t == 0) return KDA_OK;
    st = validate_rows(fn, "k", k, k_stride, kv_heads);
    if (st == KDA_OK) st = validate_rows(fn, "v", v, v_stride, kv_heads);
    if (st != KDA_OK) return st;
    const long long rows = cu ? t : (long long)t * n_seqs;
    KDA_REQUIRE(rows < 0x7fffffffLL, KDA_ERR_INVALID_ARG, "%s: more than 2^31 - 2 token rows", fn);
    KDA_REQUIRE(!fault_injected(), KDA_ERR_CUDA, "%s: injected launch failure", fn);
    RowArgs a = {(uint16_t*)k, (uint16_t*)v, k_stride, v_stride, cu, t, n_seqs,
                 {cache, table, lens, n_pages, max_pages, __builtin_ctz((unsigned)page), kv_heads}};
    const long long slots = rows / 16 + 2LL * n_seqs;
    // K and V in one warp share the search for its tokens (append and read of the
    // front end's batch: 215 us, apart 231, when this was chosen); few tokens are
    // done sooner apart.
    const unsigned apart = slots * kv_heads < 16LL * 152 ? 2 : 1;
    const dim3 grid((unsigned)((slots + kWarps - 1) / kWarps), (unsigned)kv_heads, apart);
    const dim3 threads(kWarps * 32);
    cudaStream_t s = as_stream(stream);
    if (append) {
        if (in_dtype == KDA_F16) append_kernel<true><<<grid, threads, 0, s>>>(a);
        else append_kernel<false><<<grid, threads, 0, s>>>(a);
    } else {
        if (in_dtype == KDA_F16) read_kernel<true><<<grid, threads, 0, s>>>(a);
        else read_kernel<false><<<grid, threads, 0, s>>>(a);
    }
    return launch_result(fn);
}

}  // namespace

cudaError_t status_word_kv4(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_kv4_status);
}

kda_status validate_cache(const char* fn, const void* cache, int64_t n_pages, int page,
                          const int* table, int max_pages, const int* lens, int n_seqs,
                          int kv_heads, int head_dim) {
    KDA_REQUIRE(head_dim == D, KDA_ERR_UNSUPPORTED, "%s: head_dim %d unsupported (only 128)", fn,
                head_dim);
    KDA_REQUIRE(page == 16 || page == 32 || page == 64 || page == 128 || page == 256,
                KDA_ERR_UNSUPPORTED, "%s: pages of %d tokens (only 16, 32, 64, 128, 256)", fn,
                page);
    KDA_REQUIRE(n_seqs >= 1 && kv_heads >= 1 && kv_heads <= 65535 && n_pages >= 1 &&
                    max_pages >= 1 && max_pages <= 0x7fffffff / page,
                KDA_ERR_INVALID_ARG,
                "%s: n_seqs (%d), kv_heads (%d), n_pages (%lld) and max_pages (%d) must be "
                "positive, and max_pages * page below 2^31",
                fn, n_seqs, kv_heads, (long long)n_pages, max_pages);
    KDA_REQUIRE(cache && table && lens, KDA_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    KDA_REQUIRE(aligned16(cache), KDA_ERR_INVALID_ARG, "%s: the cache must be 16-byte aligned",
                fn);
    KDA_REQUIRE((reinterpret_cast<uintptr_t>(table) & 3) == 0 &&
                    (reinterpret_cast<uintptr_t>(lens) & 3) == 0,
                KDA_ERR_INVALID_ARG, "%s: page_table and lens must be 4-byte aligned", fn);
    return KDA_OK;
}

}  // namespace kda

using namespace kda;

extern "C" kda_status kda_attn_kv4_append(const void* k, const void* v, int64_t k_row_stride,
                                          int64_t v_row_stride, int t, const int* cu_seqlens,
                                          int n_seqs, int kv_heads, int head_dim, int in_dtype,
                                          uint8_t* cache, int64_t n_pages, int page,
                                          const int* page_table, int max_pages, const int* lens,
                                          uint64_t stream) {
    return rows_call("kda_attn_kv4_append", true, const_cast<void*>(k), const_cast<void*>(v),
                     k_row_stride, v_row_stride, t, cu_seqlens, n_seqs, kv_heads, head_dim,
                     in_dtype, cache, n_pages, page, page_table, max_pages, lens, stream);
}

extern "C" kda_status kda_attn_kv4_read(void* k, void* v, int64_t k_row_stride,
                                        int64_t v_row_stride, int t, const int* cu_seqlens,
                                        int n_seqs, int kv_heads, int head_dim, int in_dtype,
                                        const uint8_t* cache, int64_t n_pages, int page,
                                        const int* page_table, int max_pages, const int* lens,
                                        uint64_t stream) {
    return rows_call("kda_attn_kv4_read", false, k, v, k_row_stride, v_row_stride, t, cu_seqlens,
                     n_seqs, kv_heads, head_dim, in_dtype, const_cast<uint8_t*>(cache), n_pages,
                     page, page_table, max_pages, lens, stream);
}
