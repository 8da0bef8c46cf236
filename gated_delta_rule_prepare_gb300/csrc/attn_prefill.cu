// Causal attention of packed prompts (kda_attn_prefill).  For query row i of a
// sequence of Lq queries and Lk keys, at position p = Lk - Lq + i, head h and
// its KV head h / (heads / kv_heads):
//     s_j = scale * q_i . k_j          for max(0, p - window + 1) <= j <= p
//     o_i = sum_j exp(s_j - lse) v_j,  lse = log sum_j exp(s_j)
// A row that sees no key gives o = 0 and lse = -inf.
#include <cmath>

#include "attn_common.h"

namespace kda {
namespace {

using namespace attn;

__device__ unsigned g_attn_status = 0;

struct PrefillArgs {
    const uint16_t *q, *k, *v;
    uint16_t* o;
    float* lse;
    const int *cu_q, *cu_k;
    long long q_stride, k_stride, v_stride, o_stride;
    int t_q, t_k, n_seqs, heads, kv_heads, window;
    float scale;
};

// Sequence n's query and key rows; false for offsets outside the arrays.
struct Span {
    long long q0, k0;
    int lq, lk;
};
__device__ __forceinline__ bool sequence_span(const PrefillArgs& a, int n, Span& s) {
    if (!a.cu_q) {
        s = {(long long)n * a.t_q, (long long)n * a.t_k, a.t_q, a.t_k};
        return true;
    }
    const int q0 = __ldg(a.cu_q + n), q1 = __ldg(a.cu_q + n + 1);
    const int k0 = __ldg(a.cu_k + n), k1 = __ldg(a.cu_k + n + 1);
    s = {q0, k0, q1 - q0, k1 - k0};
    return q0 >= 0 && q0 <= q1 && q1 <= a.t_q && k0 >= 0 && k0 <= k1 && k1 <= a.t_k;
}

// One (row, head) per warp, 4 channels a lane: one pass over the row's keys
// with the running maximum and sum of the softmax.
template <bool F16>
__device__ __forceinline__ void attend_row(const PrefillArgs& a, const Span& s, int i, int h) {
    const int lane = threadIdx.x & 31;
    const int hk = h / (a.heads / a.kv_heads);
    const int p = s.lk - s.lq + i;
    const int first = a.window ? max(0, p - a.window + 1) : 0;
    const uint2 qb = __ldg(reinterpret_cast<const uint2*>(a.q + (s.q0 + i) * a.q_stride +
                                                          h * D + 4 * lane));
    const float c = a.scale * kLog2e;
    const float2 q01 = widen2<F16>(qb.x), q23 = widen2<F16>(qb.y);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const uint16_t* kp = a.k + s.k0 * a.k_stride + hk * D + 4 * lane;
    const uint16_t* vp = a.v + s.k0 * a.v_stride + hk * D + 4 * lane;
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
    *reinterpret_cast<uint2*>(a.o + (s.q0 + i) * a.o_stride + h * D + 4 * lane) = out;
    if (a.lse && lane == 0)
        a.lse[(s.q0 + i) * a.heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <bool F16>
__global__ void __launch_bounds__(256) attn_rows_kernel(PrefillArgs a, long long units) {
    const long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (blockIdx.x == 0 && threadIdx.x < 32 && a.cu_q &&
        !(warp_offsets_ok(a.cu_q, a.n_seqs, a.t_q) && warp_offsets_ok(a.cu_k, a.n_seqs, a.t_k)) &&
        threadIdx.x == 0)
        atomicOr(&g_attn_status, STATUS_BAD_CU_SEQLENS);
    if (u >= units) return;
    const long long row = u / a.heads;
    const int h = (int)(u - row * a.heads);
    const int n = a.cu_q ? warp_find_last(a.n_seqs, row, [&](int i) { return __ldg(a.cu_q + i); })
                         : (int)(row / a.t_q);
    Span s;
    if (!sequence_span(a, n, s) || row < s.q0 || row >= s.q0 + s.lq) return;
    attend_row<F16>(a, s, (int)(row - s.q0), h);
}

}  // namespace

cudaError_t read_and_clear_status_attn(unsigned* out) {
    const unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_attn_status, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(unsigned));
    return e;
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
    if (rows < 0 || n_seqs < 1 || heads < 1 || kv_heads < 1 || heads % kv_heads) return 0;
    return 256;
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
    PrefillArgs a = {(const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v, (uint16_t*)o,
                     lse, cu_seqlens_q, cu_seqlens_k, q_row_stride, k_row_stride, v_row_stride,
                     o_row_stride, t_q, t_k, n_seqs, heads, kv_heads, window, scale};
    const long long units = rows_q * heads;
    KDA_REQUIRE((units + 7) / 8 < 0x7fffffffLL, KDA_ERR_INVALID_ARG, "%s: problem too large", fn);
    const size_t need = kda_attn_prefill_workspace_size(rows_q, n_seqs, heads, kv_heads);
    KDA_REQUIRE(workspace && workspace_bytes >= need, KDA_ERR_WORKSPACE,
                "%s: workspace of %zu B, %zu B needed", fn, workspace ? workspace_bytes : 0, need);
    KDA_REQUIRE(aligned16(workspace), KDA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned",
                fn);
    KDA_REQUIRE(!fault_injected(), KDA_ERR_CUDA, "%s: injected launch failure", fn);
    const dim3 grid((unsigned)((units + 7) / 8));
    if (in_dtype == KDA_F16)
        attn_rows_kernel<true><<<grid, 256, 0, as_stream(stream)>>>(a, units);
    else
        attn_rows_kernel<false><<<grid, 256, 0, as_stream(stream)>>>(a, units);
    return launch_result(fn);
}
