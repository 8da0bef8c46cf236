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
// Both kernels give one warp 16 tokens of one head of K or of V: one group of
// the cache, 1024 bytes of codes, staged in shared memory so that global
// memory sees 16-byte accesses on both sides.  Memory-bound: 512 + 144 bytes
// per (token, head).
#include "attn_common.h"

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

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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

// The code of x near a border between two codes, or where 1/s overflows:
// compares x with the borders m + (c + 0.5) s.  c + 0.5 has 5 bits and s has 8,
// so (c + 0.5) s is exact; t + e is x - m exactly (the rounded difference and
// what it lost), and the fused multiply-add gets the comparison's sign right.
__device__ __noinline__ uint32_t code_at_border(float x, float m, float s) {
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
// bits 4x.
template <bool F16>
__device__ __forceinline__ uint32_t codes8(const uint4& raw, float m, float s, float inv) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t out = 0;
    bool near = !(inv < 1e37f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = widen2<F16>(w[i]);
        const float a = (x.x - m) * inv, b = (x.y - m) * inv;
        const float ra = rintf(a), rb = rintf(b);
        // the quotient is good to 2^-18: only these can be on the wrong side
        near |= fabsf(a - ra) > 0.4999f || fabsf(b - rb) > 0.4999f;
        out |= min((uint32_t)ra, 15u) << (8 * i) | min((uint32_t)rb, 15u) << (8 * i + 4);
    }
    if (near) {
        out = 0;
        for (int i = 0; i < 4; ++i) {
            const float2 x = widen2<F16>(w[i]);
            out |= code_at_border(x.x, m, s) << (8 * i) |
                   code_at_border(x.y, m, s) << (8 * i + 4);
        }
    }
    return s > 0.f ? out : 0u;
}

// grid (ceil(slots / 4), kv_heads, 2): z = 0 writes K, z = 1 V.  A half-warp
// loads a token row of 128 channels, 16 bytes a lane, all sixteen tokens of
// the group in flight; minimum and maximum over 64 channels are 8-lane
// shuffles.
template <bool F16>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(RowArgs a) {
    __shared__ __align__(16) uint8_t stage[kWarps][kStage];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    check_offsets(a);
    Slot s;
    if (!find_slot(a, (long long)blockIdx.x * kWarps + warp, s)) return;  // whole warps
    const int h = blockIdx.y;
    const bool is_v = blockIdx.z;
    uint8_t* block = a.c.block(s.n, s.pos, h);
    if (!block) {
        if (lane == 0) atomicOr(&g_kv4_status, STATUS_BAD_PAGES);
        return;
    }
    if (is_v) block += part_bytes(a.c.page());
    const long long stride = is_v ? a.v_stride : a.k_stride;
    const uint16_t* src = (is_v ? a.v : a.k) + h * D;
    const int hw = lane >> 4, c = lane & 15, b = c >> 1;
    const int t0 = s.pos & 15;  // first token of the group that is written
    uint4 raw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int tok = 2 * j + hw;
        const bool mine = tok >= t0 && tok < t0 + s.count;
        raw[j] = mine ? __ldg(reinterpret_cast<const uint4*>(
                            src + (s.row + tok - t0) * stride + 8 * c))
                      : make_uint4(0, 0, 0, 0);
    }
    const int in_page = s.pos & (a.c.page() - 1) & ~15;
    uint8_t* par = block + a.c.page() * 64 + (long long)in_page * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int tok = 2 * j + hw;
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
        float lo, hi;
        {
            const float2 x = widen2<F16>(w[0]);
            lo = min_nan(x.x, x.y);
            hi = max_nan(x.x, x.y);
        }
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const float2 x = widen2<F16>(w[i]);
            lo = min_nan(lo, min_nan(x.x, x.y));
            hi = max_nan(hi, max_nan(x.x, x.y));
        }
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) {
            lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
            hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        }
        uint32_t mb = bf16_down(lo);
        const float m = __uint_as_float(mb << 16);
        // both rounded up: at or above the real quotient, and equal to it
        // where it is a BF16 number
        const float q = __fdiv_ru(__fsub_ru(hi, m), 15.f);
        uint32_t sb = bf16_up(q);
        // an infinity or a NaN in the group: every value of it reads as NaN
        const bool bad = !(q < 3e38f) || !(fabsf(m) < INFINITY);
        if (bad) mb = sb = 0x7fffu;
        const float sc = bad ? 0.f : __uint_as_float(sb << 16);
        const uint32_t own = codes8<F16>(raw[j], bad ? 0.f : m, sc, 1.f / sc);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
        // channels 16 b + x (low bits, the even lane's) and 16 b + 8 + x
        const uint32_t even = lane & 1 ? other : own, odd = lane & 1 ? own : other;
        const int x0 = (lane & 1) * 4;  // the even lane stores x = 0..3, the odd one 4..7
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = x0 + i;
            const uint32_t byte = (even >> (4 * x) & 15u) | (odd >> (4 * x) & 15u) << 4;
            const int hi8 = tok >> 3, lo8 = tok & 7;
            const int at = 512 * (b >> 2) + 4 * (b & 3) +
                           (is_v ? 16 * (4 * x + (lo8 >> 1)) + 2 * (lo8 & 1) + hi8
                                 : 16 * (4 * lo8 + (x >> 1)) + 2 * (x & 1) + hi8);
            stage[warp][staged(at)] = (uint8_t)byte;
        }
        if ((c & 7) == 0 && tok >= t0 && tok < t0 + s.count)
            *reinterpret_cast<uint32_t*>(par + tok * 8 + (c >> 3) * 4) = sb | mb << 16;
    }
    __syncwarp();
    uint8_t* codes = block + (long long)in_page * 64;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int at = half * 512 + lane * 16;
        const uint4 v = *reinterpret_cast<const uint4*>(&stage[warp][staged(at)]);
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

// grid as append_kernel.  A lane turns 8 channels of a token into 16 bytes.
template <bool F16>
__global__ void __launch_bounds__(kWarps * 32) read_kernel(RowArgs a) {
    __shared__ __align__(16) uint8_t stage[kWarps][kStage];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    check_offsets(a);
    Slot s;
    if (!find_slot(a, (long long)blockIdx.x * kWarps + warp, s)) return;
    const int h = blockIdx.y;
    const bool is_v = blockIdx.z;
    const uint8_t* block = a.c.block(s.n, s.pos, h);
    if (!block && lane == 0) atomicOr(&g_kv4_status, STATUS_BAD_PAGES);
    const long long stride = is_v ? a.v_stride : a.k_stride;
    uint16_t* dst = (is_v ? a.v : a.k) + h * D;
    const int hw = lane >> 4, c = lane & 15, b = c >> 1;
    const int t0 = s.pos & 15;
    const int in_page = s.pos & (a.c.page() - 1) & ~15;
    const uint8_t* par = nullptr;
    if (block) {
        if (is_v) block += part_bytes(a.c.page());
        par = block + a.c.page() * 64 + (long long)in_page * 8 + (c >> 3) * 4;
        const uint8_t* codes = block + (long long)in_page * 64;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int at = half * 512 + lane * 16;
            *reinterpret_cast<uint4*>(&stage[warp][staged(at)]) =
                __ldg(reinterpret_cast<const uint4*>(codes + at));
        }
    }
    __syncwarp();
    const uint8_t* mine = &stage[warp][staged(512 * (b >> 2)) + 4 * (b & 3)];
    const int sh = 4 * (lane & 1);
    // One token: byte_of(x) holds the code of its channel x = 0..7 of this lane.
    auto put = [&](int tok, auto byte_of) {
        if (tok < t0 || tok >= t0 + s.count) return;
        // a page that is not there reads as NaN
        const uint32_t p = par ? __ldg(reinterpret_cast<const uint32_t*>(par + tok * 8))
                               : 0x7fff7fffu;
        const float sc = __uint_as_float(p << 16), m = __uint_as_float(p & 0xffff0000u);
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = (float)(byte_of(2 * i) >> sh & 15u);
            const float hi = (float)(byte_of(2 * i + 1) >> sh & 15u);
            out[i] = narrow2<F16>(fmaf(sc, lo, m), fmaf(sc, hi, m));
        }
        *reinterpret_cast<uint4*>(dst + (s.row + tok - t0) * stride + 8 * c) =
            make_uint4(out[0], out[1], out[2], out[3]);
    };
    if (!is_v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int g = 2 * j + hw;  // tokens g and g + 8 share words t = 0..3
            uint32_t w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                w[t] = *reinterpret_cast<const uint32_t*>(mine + 16 * (4 * g + t));
#pragma unroll
            for (int i = 0; i < 2; ++i)
                put(g + 8 * i, [&](int x) { return w[x >> 1] >> (16 * (x & 1) + 8 * i); });
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = 2 * j + hw;  // tokens 2t, 2t + 1, 2t + 8, 2t + 9 share words x = 0..7
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x)
                w[x] = *reinterpret_cast<const uint32_t*>(mine + 16 * (4 * x + t));
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    put(2 * t + e + 8 * i, [&](int x) { return w[x] >> (16 * e + 8 * i); });
        }
    }
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
    const dim3 grid((unsigned)((slots + kWarps - 1) / kWarps), (unsigned)kv_heads, 2);
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

cudaError_t read_and_clear_status_kv4(unsigned* out) {
    const unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_kv4_status, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_kv4_status, &zero, sizeof(unsigned));
    return e;
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
