// What the linear-attention kernels share: the arguments of a call and a
// sequence's rows.
#pragma once

#include "attn_common.h"

namespace kda {
namespace lin {

struct Args {
    const float* state_in;  // null: zeros
    float* state_out;       // null: not wanted
    const uint16_t *q, *k, *v;
    const float* g;
    uint16_t* o;
    const int* cu;  // null: n_seqs sequences of t rows, t_pad rows apart
    int t, t_pad, n_seqs, heads, qk_heads;
    long long q_stride, k_stride, v_stride, g_stride, o_stride;
    float scale;

    __device__ __forceinline__ int qk_head(int h) const { return h / (heads / qk_heads); }
};

// The smallest exponent a decay keeps: e^-110 of any FP32 number is below 2^-30,
// and e^-104 is below FP32's smallest.  Running sums of clamped values stay finite,
// so that differences of them are no NaN; a NaN stays one.
constexpr float kLeastDecay = -110.f;
__device__ __forceinline__ float clamp_decay(float g) { return g < kLeastDecay ? kLeastDecay : g; }

struct Rows {
    long long first;
    int count;
};
// Sequence n's rows; false for offsets outside the arrays.
__device__ __forceinline__ bool sequence_rows(const Args& a, int n, Rows& r) {
    if (!a.cu) {
        r = {(long long)n * a.t_pad, a.t};
        return true;
    }
    const int c0 = __ldg(a.cu + n), c1 = __ldg(a.cu + n + 1);
    r = {c0, c1 - c0};
    return c0 >= 0 && c0 <= c1 && c1 <= a.t;
}

}  // namespace lin

// The row walk (lin_walk.cu): any number of rows of each sequence, one after the
// other.
struct LinSnaps {
    float* p[KDA_MAX_K];
    int n;
};
void launch_lin_walk(const lin::Args& a, bool f16, const LinSnaps& snaps, cudaStream_t s);

// The chunked form (lin_prefill.cu).
size_t lin_chunked_workspace_bytes(long long rows, int n_seqs, int heads);
kda_status launch_lin_chunked(const lin::Args& a, bool f16, void* workspace, cudaStream_t s);

}  // namespace kda
