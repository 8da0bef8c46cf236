// Attention of 1..8 query rows per sequence over the paged 4-bit cache
// (kda_attn_kv4_decode).
#include <cmath>

#include "attn_common.h"

namespace kda {
namespace {

using namespace attn;

__device__ unsigned g_decode_status = 0;

struct DecodeArgs {
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    int n_seqs, krows, heads, window;
    float scale;
    Cache c;
};

// Four channels 4l .. 4l + 3 of a token.
__device__ __forceinline__ float4 token4(const uint8_t* part, int page, int at, bool is_v) {
    const int lane = threadIdx.x & 31, ch = 4 * lane;
    const uint8_t* group = part + (at >> 4) * 1024;
    const int tok = at & 15, a = ch >> 6, b = ch >> 4 & 3, j = ch >> 3 & 1;
    float r[4];
    const float2 sm = widen2<false>(__ldg(reinterpret_cast<const uint32_t*>(
        part + page * 64 + at * 8 + a * 4)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int x = (ch & 7) + i;
        const int t8 = tok & 7;
        const int byte = 512 * a + 4 * b + (tok >> 3) +
                         (is_v ? 16 * (4 * x + (t8 >> 1)) + 2 * (t8 & 1)
                               : 16 * (4 * t8 + (x >> 1)) + 2 * (x & 1));
        r[i] = fmaf(sm.x, (float)(__ldg(group + byte) >> (4 * j) & 15), sm.y);
    }
    return make_float4(r[0], r[1], r[2], r[3]);
}

// One (sequence, row, head) per warp.
template <bool F16>
__global__ void __launch_bounds__(256) decode_rows_kernel(DecodeArgs a, long long units) {
    const long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (u >= units) return;
    const int lane = threadIdx.x & 31;
    const int h = (int)(u % a.heads);
    const long long row = u / a.heads;
    const int n = (int)(row / a.krows), i = (int)(row % a.krows);
    const int hk = h / (a.heads / a.c.kv_heads), page = a.c.page();
    int len = __ldg(a.c.lens + n);
    if (len < 0 || len > a.c.max_pages * page) {
        if (lane == 0) atomicOr(&g_decode_status, STATUS_BAD_PAGES);
        len = 0;
    }
    const int p = len - a.krows + i;
    const int first = a.window ? max(0, p - a.window + 1) : 0;
    const uint2 qb = __ldg(reinterpret_cast<const uint2*>(a.q + u * D + 4 * lane));
    const float2 q01 = widen2<F16>(qb.x), q23 = widen2<F16>(qb.y);
    const float c = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = first; j <= p; ++j) {
        const uint8_t* block = a.c.block(n, j, hk);
        if (!block) {
            if (lane == 0) atomicOr(&g_decode_status, STATUS_BAD_PAGES);
            continue;
        }
        const int at = j & (page - 1);
        const float4 k = token4(block, page, at, false);
        float d = q01.x * k.x;
        d = fmaf(q01.y, k.y, d);
        d = fmaf(q23.x, k.z, d);
        d = fmaf(q23.y, k.w, d);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        d *= c;
        const float m2 = fmaxf(m, d);
        const float shift = m2 == -INFINITY ? 0.f : m2;
        const float keep = exp2f(m - shift), w = exp2f(d - shift);
        const float4 v = token4(block + part_bytes(page), page, at, true);
        l = fmaf(l, keep, w);
        o.x = fmaf(o.x, keep, w * v.x);
        o.y = fmaf(o.y, keep, w * v.y);
        o.z = fmaf(o.z, keep, w * v.z);
        o.w = fmaf(o.w, keep, w * v.w);
        m = m2;
    }
    const float r = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(a.o + u * D + 4 * lane) =
        make_uint2(narrow2<F16>(o.x * r, o.y * r), narrow2<F16>(o.z * r, o.w * r));
    if (a.lse && lane == 0) a.lse[u] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
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

extern "C" size_t kda_attn_kv4_workspace_size(int n_seqs, int krows, int heads, int kv_heads) {
    if (n_seqs < 1 || krows < 1 || krows > KDA_MAX_K || heads < 1 || kv_heads < 1 || heads % kv_heads) return 0;
    return 256;
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
    const long long units = (long long)n_seqs * krows * heads;
    KDA_REQUIRE((units + 7) / 8 < 0x7fffffffLL, KDA_ERR_INVALID_ARG, "%s: problem too large", fn);
    const size_t need = kda_attn_kv4_workspace_size(n_seqs, krows, heads, kv_heads);
    KDA_REQUIRE(workspace && workspace_bytes >= need, KDA_ERR_WORKSPACE,
                "%s: workspace of %zu B, %zu B needed", fn, workspace ? workspace_bytes : 0, need);
    KDA_REQUIRE(aligned16(workspace), KDA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned",
                fn);
    KDA_REQUIRE(!fault_injected(), KDA_ERR_CUDA, "%s: injected launch failure", fn);
    DecodeArgs a = {(const uint16_t*)q, (uint16_t*)o, lse, n_seqs, krows, heads, window, scale,
                    {const_cast<uint8_t*>(cache), page_table, lens, n_pages, max_pages,
                     __builtin_ctz((unsigned)page), kv_heads}};
    const dim3 grid((unsigned)((units + 7) / 8));
    if (in_dtype == KDA_F16)
        decode_rows_kernel<true><<<grid, 256, 0, as_stream(stream)>>>(a, units);
    else
        decode_rows_kernel<false><<<grid, 256, 0, as_stream(stream)>>>(a, units);
    return launch_result(fn);
}
