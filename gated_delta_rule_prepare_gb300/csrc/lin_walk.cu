// Linear attention with a decay for each head, token by token: kda_lin_decode, and
// kda_lin_prefill's short sequences.  Per head and token
//     S[i][j] <- exp(g) S[i][j] + k[i] v[j],     o[j] = scale * sum_i q[i] S[i][j]
//
// Bound by the state: 64 KB a head in and out, and 64 KB more for each snapshot,
// against 1 KB of rows.  A CTA of 256 threads has J value channels of one
// head (columns of S do not meet), each thread a few rows of four columns in
// registers for all tokens.  J = 128 reads whole state rows; with few heads
// J = 32 spreads each over four multiprocessors.
//
// A token's partial sums over i go through shared memory in a fixed order, and its
// inputs are staged while the last one's step runs, one barrier a token.  The same
// code runs whatever the number of tokens, and every operation is explicitly
// rounded, so k tokens in one call give the bits of k calls.
//
// 64 sequences of 32 heads, one token (270 MB): 44.0 us, 6.2 TB/s.  3 sequences of 16 heads,
// four tokens with their states (19 MB): 7.5 us a call.
#include "lin_attn.h"

namespace kda {
namespace {

using namespace attn;
using lin::Args;

__device__ unsigned g_lin_walk_status = 0;

constexpr int kThreads = 256;

template <bool F16>
__device__ __forceinline__ float widen(uint16_t u) {
    if constexpr (F16) return __half2float(__ushort_as_half(u));
    else return __uint_as_float((uint32_t)u << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t narrow(float x) {
    return (uint16_t)(narrow2<F16>(x, 0.f) & 0xffffu);
}

template <bool F16, int J>
__global__ void __launch_bounds__(kThreads)
lin_walk_kernel(Args a, LinSnaps snaps) {
    constexpr int kCols = J / 4;               // threads across the columns
    constexpr int kGroups = kThreads / kCols;  // row groups
    constexpr int kRows = D / kGroups;         // state rows a thread
    constexpr int kPart = 8;                   // partial sums of a column: one a warp
    struct alignas(16) Token {
        float q[D], k[D], v[J], decay;
    };
    __shared__ Token token[2];
    __shared__ __align__(16) float part[2][kPart][J];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_release();
    if (a.cu && blockIdx.x == 0 && warp == 0 && !warp_offsets_ok(a.cu, a.n_seqs, a.t) && lane == 0)
        atomicOr(&g_lin_walk_status, STATUS_BAD_CU_SEQLENS);
    const int nh = blockIdx.x / (D / J), j0 = (blockIdx.x - nh * (D / J)) * J;
    const int n = nh / a.heads, h = nh - n * a.heads, hq = a.qk_head(h);
    lin::Rows rows;
    if (!sequence_rows(a, n, rows)) return;

    // A thread's inputs of a token: channel tid of q (threads below 128) or of k, and
    // of v one of the first J threads'.
    const uint16_t* qk = tid < D ? a.q + rows.first * a.q_stride + hq * D + tid
                                 : a.k + rows.first * a.k_stride + hq * D + tid - D;
    const long long qk_stride = tid < D ? a.q_stride : a.k_stride;
    const uint16_t* vp = a.v + rows.first * a.v_stride + h * D + j0 + tid;
    const float* gp = a.g + rows.first * a.g_stride + h;
    auto stage = [&](Token& to, int t) {
        const float x = widen<F16>(__ldg(qk + t * qk_stride));
        (tid < D ? to.q[tid] : to.k[tid - D]) = tid < D ? __fmul_rn(a.scale, x) : x;
        if (tid < J) to.v[tid] = widen<F16>(__ldg(vp + t * a.v_stride));
        if (tid == kThreads - 1) to.decay = expf(__ldg(gp + t * a.g_stride));
    };
    if (rows.count > 0) stage(token[0], 0);

    const int group = tid / kCols, col = (tid - group * kCols) * 4;
    const size_t at = (size_t)nh * D * D + (size_t)group * kRows * D + j0 + col;
    float4 s[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        s[r] = a.state_in ? __ldcs(reinterpret_cast<const float4*>(a.state_in + at + r * D))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    auto store = [&](float* to) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            __stcs(reinterpret_cast<float4*>(to + at + r * D), s[r]);
    };
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < rows.count; ++t) {
        const Token& x = token[t & 1];
        const float4 v = *reinterpret_cast<const float4*>(x.v + col);
        const float decay = x.decay;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float k = x.k[group * kRows + r], q = x.q[group * kRows + r];
            s[r].x = __fmaf_rn(k, v.x, __fmul_rn(decay, s[r].x));
            s[r].y = __fmaf_rn(k, v.y, __fmul_rn(decay, s[r].y));
            s[r].z = __fmaf_rn(k, v.z, __fmul_rn(decay, s[r].z));
            s[r].w = __fmaf_rn(k, v.w, __fmul_rn(decay, s[r].w));
            sum.x = __fmaf_rn(q, s[r].x, sum.x);
            sum.y = __fmaf_rn(q, s[r].y, sum.y);
            sum.z = __fmaf_rn(q, s[r].z, sum.z);
            sum.w = __fmaf_rn(q, s[r].w, sum.w);
        }
        // row groups of one warp, then of all
#pragma unroll
        for (int off = kCols; off < 32; off <<= 1) {
            sum.x = __fadd_rn(sum.x, __shfl_xor_sync(0xffffffffu, sum.x, off));
            sum.y = __fadd_rn(sum.y, __shfl_xor_sync(0xffffffffu, sum.y, off));
            sum.z = __fadd_rn(sum.z, __shfl_xor_sync(0xffffffffu, sum.z, off));
            sum.w = __fadd_rn(sum.w, __shfl_xor_sync(0xffffffffu, sum.w, off));
        }
        if (lane < kCols) *reinterpret_cast<float4*>(&part[t & 1][warp][col]) = sum;
        if (t + 1 < rows.count) stage(token[(t + 1) & 1], t + 1);
        __syncthreads();
        if (tid < J) {
            float o = part[t & 1][0][tid];
#pragma unroll
            for (int w = 1; w < kPart; ++w) o = __fadd_rn(o, part[t & 1][w][tid]);
            a.o[(rows.first + t) * a.o_stride + h * D + j0 + tid] = narrow<F16>(o);
        }
        if (t < snaps.n) store(snaps.p[t]);
    }
    if (a.state_out) store(a.state_out);
}

}  // namespace

cudaError_t status_word_lin_walk(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_lin_walk_status);
}

void launch_lin_walk(const Args& a, bool f16, const LinSnaps& snaps, cudaStream_t s) {
    // quarters of heads while there are two for each multiprocessor at most (32 heads: 2.5 us,
    // whole ones 3.2; 64, with four snapshots: 6.4, and 8.4; 128: 4.5, and 3.6)
    const int chains = a.n_seqs * a.heads;
    const bool wide = 2 * chains > 152;
    auto kernel = wide ? lin_walk_kernel<false, 128> : lin_walk_kernel<false, 32>;
    if (f16) kernel = wide ? lin_walk_kernel<true, 128> : lin_walk_kernel<true, 32>;
    launch_pdl(kernel, dim3((unsigned)chains * (wide ? 1 : 4)), dim3(kThreads), 0, s, a, snaps);
}

}  // namespace kda

using namespace kda;

namespace {

// Checks that both calls make; rows: token rows of the arrays.
kda_status check_lin(const char* fn, const lin::Args& a, long long rows, int head_dim,
                     int in_dtype) {
    KDA_REQUIRE(head_dim == D, KDA_ERR_UNSUPPORTED, "%s: head_dim %d unsupported (only 128)", fn,
                head_dim);
    KDA_REQUIRE(in_dtype == KDA_F32 || in_dtype == KDA_BF16 || in_dtype == KDA_F16,
                KDA_ERR_INVALID_ARG, "%s: in_dtype %d is not a kda_dtype", fn, in_dtype);
    KDA_REQUIRE(in_dtype != KDA_F32, KDA_ERR_UNSUPPORTED, "%s: FP32 inputs are not built", fn);
    KDA_REQUIRE(a.n_seqs >= 1, KDA_ERR_INVALID_ARG, "%s: n_seqs (%d) must be >= 1", fn, a.n_seqs);
    KDA_REQUIRE(a.heads >= 1 && a.qk_heads >= 1 && a.heads % a.qk_heads == 0, KDA_ERR_INVALID_ARG,
                "%s: heads (%d) must be a positive multiple of qk_heads (%d)", fn, a.heads,
                a.qk_heads);
    KDA_REQUIRE((long long)a.n_seqs * a.heads <= 0x1fffffffLL, KDA_ERR_INVALID_ARG,
                "%s: n_seqs * heads too large", fn);
    KDA_REQUIRE(rows < 0x7fffffffLL, KDA_ERR_INVALID_ARG, "%s: more than 2^31 - 2 token rows", fn);
    KDA_REQUIRE(isfinite(a.scale), KDA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    KDA_REQUIRE(aligned16(a.state_in) && aligned16(a.state_out), KDA_ERR_INVALID_ARG,
                "%s: the states must be 16-byte aligned", fn);
    if (rows == 0) return KDA_OK;
    kda_status st = validate_rows(fn, "q", a.q, a.q_stride, a.qk_heads);
    if (st == KDA_OK) st = validate_rows(fn, "k", a.k, a.k_stride, a.qk_heads);
    if (st == KDA_OK) st = validate_rows(fn, "v", a.v, a.v_stride, a.heads);
    if (st == KDA_OK) st = validate_rows(fn, "o", a.o, a.o_stride, a.heads);
    if (st != KDA_OK) return st;
    KDA_REQUIRE(a.g, KDA_ERR_INVALID_ARG, "%s: null pointer argument (g)", fn);
    KDA_REQUIRE((reinterpret_cast<uintptr_t>(a.g) & 3) == 0, KDA_ERR_INVALID_ARG,
                "%s: g must be 4-byte aligned", fn);
    KDA_REQUIRE(a.g_stride == 0 || a.g_stride >= a.heads, KDA_ERR_INVALID_ARG,
                "%s: g row stride %lld must be 0 or >= heads", fn, a.g_stride);
    return KDA_OK;
}

}  // namespace

extern "C" kda_status kda_lin_decode(const float* state_in, float* state_out, const void* q,
                                     const void* k, const void* v, const float* g, void* o,
                                     int n_seqs, int krows, int heads, int qk_heads, int head_dim,
                                     int in_dtype, int64_t q_row_stride, int64_t k_row_stride,
                                     int64_t v_row_stride, int64_t g_row_stride,
                                     int64_t o_row_stride, float scale, float* const* snapshots,
                                     int n_snap, uint64_t stream) {
    const char* fn = "kda_lin_decode";
    KDA_REQUIRE(krows >= 1 && krows <= KDA_MAX_K, KDA_ERR_INVALID_ARG,
                "%s: k = %d outside [1, %d]", fn, krows, KDA_MAX_K);
    const lin::Args a = {state_in, state_out, (const uint16_t*)q, (const uint16_t*)k,
                         (const uint16_t*)v, g, (uint16_t*)o, nullptr, krows, krows, n_seqs,
                         heads, qk_heads, q_row_stride, k_row_stride, v_row_stride, g_row_stride,
                         o_row_stride, scale};
    const kda_status st = check_lin(fn, a, (long long)n_seqs * krows, head_dim, in_dtype);
    if (st != KDA_OK) return st;
    KDA_REQUIRE(n_snap >= 0 && n_snap <= krows, KDA_ERR_INVALID_ARG,
                "%s: n_snap = %d outside [0, k = %d]", fn, n_snap, krows);
    KDA_REQUIRE(n_snap == 0 || snapshots, KDA_ERR_INVALID_ARG,
                "%s: snapshots is NULL with n_snap = %d", fn, n_snap);
    LinSnaps snaps = {};
    snaps.n = n_snap;
    for (int t = 0; t < n_snap; ++t) {
        KDA_REQUIRE(snapshots[t] && aligned16(snapshots[t]), KDA_ERR_INVALID_ARG,
                    "%s: snapshot %d is NULL or not 16-byte aligned", fn, t);
        KDA_REQUIRE(snapshots[t] != state_in && snapshots[t] != state_out, KDA_ERR_INVALID_ARG,
                    "%s: snapshot %d aliases the state", fn, t);
        snaps.p[t] = snapshots[t];
    }
    KDA_REQUIRE(!fault_injected(), KDA_ERR_CUDA, "%s: injected launch failure", fn);
    launch_lin_walk(a, in_dtype == KDA_F16, snaps, as_stream(stream));
    return launch_result(fn);
}

extern "C" size_t kda_lin_prefill_workspace_size(int64_t rows, int n_seqs, int heads) {
    if (rows < 0 || rows >= 0x7fffffffLL || n_seqs < 1 || heads < 1 ||
        (long long)n_seqs * heads > 0x1fffffffLL)
        return 0;
    return lin_chunked_workspace_bytes(rows, n_seqs, heads);
}

extern "C" kda_status kda_lin_prefill(const float* state_in, float* state_out, const void* q,
                                      const void* k, const void* v, const float* g, void* o, int t,
                                      int t_pad, const int* cu_seqlens, int n_seqs, int heads,
                                      int qk_heads, int head_dim, int in_dtype,
                                      int64_t q_row_stride, int64_t k_row_stride,
                                      int64_t v_row_stride, int64_t g_row_stride,
                                      int64_t o_row_stride, float scale, void* workspace,
                                      size_t workspace_bytes, uint64_t stream) {
    const char* fn = "kda_lin_prefill";
    KDA_REQUIRE(t >= 0 && t_pad >= t && (!cu_seqlens || t_pad == t), KDA_ERR_INVALID_ARG,
                "%s: t = %d, t_pad = %d (t <= t_pad, equal for packed rows)", fn, t, t_pad);
    const long long rows = cu_seqlens ? t : (long long)t_pad * n_seqs;
    const lin::Args a = {state_in, state_out, (const uint16_t*)q, (const uint16_t*)k,
                         (const uint16_t*)v, g, (uint16_t*)o, cu_seqlens, t, t_pad, n_seqs, heads,
                         qk_heads, q_row_stride, k_row_stride, v_row_stride, g_row_stride,
                         o_row_stride, scale};
    const kda_status st = check_lin(fn, a, t == 0 ? 0 : rows, head_dim, in_dtype);
    if (st != KDA_OK) return st;
    KDA_REQUIRE((reinterpret_cast<uintptr_t>(cu_seqlens) & 3) == 0, KDA_ERR_INVALID_ARG,
                "%s: cu_seqlens must be 4-byte aligned", fn);
    const size_t need = lin_chunked_workspace_bytes(rows, n_seqs, heads);
    KDA_REQUIRE(workspace && workspace_bytes >= need, KDA_ERR_WORKSPACE,
                "%s: workspace of %zu B, %zu B needed", fn, workspace ? workspace_bytes : 0, need);
    KDA_REQUIRE(aligned16(workspace), KDA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned",
                fn);
    KDA_REQUIRE(!fault_injected(), KDA_ERR_CUDA, "%s: injected launch failure", fn);
    const bool f16 = in_dtype == KDA_F16;
    if (t == 0 || (!cu_seqlens && t <= KDA_MAX_K)) {
        launch_lin_walk(a, f16, LinSnaps{}, as_stream(stream));
        return launch_result(fn);
    }
    return launch_lin_chunked(a, f16, workspace, as_stream(stream));
}
