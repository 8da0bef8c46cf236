// What the full-attention kernels share: 16-bit element conversion, the search
// that finds a packed row's sequence, and the layout of the 4-bit cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kda_common.h"

namespace kda {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Two 16-bit elements (BF16, or FP16 where F16) to FP32 and back (to nearest).
template <bool F16>
__device__ __forceinline__ float2 widen2(uint32_t u) {
    if constexpr (F16) {
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    } else {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
}
template <bool F16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// The last n in [0, n_seqs) with key(n) <= x, for a non-decreasing key with
// key(0) <= x; the whole warp searches, 32 probes a step, so up to 1024
// sequences take two dependent loads.
template <class Key>
__device__ __forceinline__ int warp_find_last(int n_seqs, long long x, Key key) {
    const int lane = threadIdx.x & 31;
    int lo = 0, count = n_seqs;
    while (count > 1) {
        const int step = (count + 31) / 32;
        const int at = lane * step;
        const unsigned yes = __ballot_sync(0xffffffffu, at < count && key(lo + at) <= x);
        const int hit = yes ? 31 - __clz(yes) : 0;
        lo += hit * step;
        count = min(step, count - hit * step);
    }
    return lo;
}

// Whether a device-side offset list is one of `t` packed rows: starts at 0,
// never falls, ends at t.  One warp looks at all of it.
__device__ __forceinline__ bool warp_offsets_ok(const int* cu, int n_seqs, int t) {
    const int lane = threadIdx.x & 31;
    bool ok = true;
    for (int i = lane; i <= n_seqs; i += 32) {
        const int c = __ldg(cu + i);
        if (i == 0 && c != 0) ok = false;
        if (i == n_seqs ? c != t : __ldg(cu + i + 1) < c) ok = false;
    }
    return __all_sync(0xffffffffu, ok);
}

// The part of it that a numbering of the rows rests on: never falls, stays within
// 0..t.
__device__ __forceinline__ bool warp_offsets_rise(const int* cu, int n_seqs, int t) {
    bool ok = true;
    for (int i = threadIdx.x & 31; i <= n_seqs; i += 32) {
        const int c = __ldg(cu + i);
        if (c < 0 || c > t || (i < n_seqs && __ldg(cu + i + 1) < c)) ok = false;
    }
    return __all_sync(0xffffffffu, ok);
}

// ---------------------------------------------------------------- 4-bit cache
// Bytes of one token's K and V, and where the V half of a block of `page`
// tokens of one KV head starts (K codes, K parameters, V codes, V parameters).
constexpr int kTokenBytes = KDA_KV4_TOKEN_BYTES;
__host__ __device__ inline int part_bytes(int page) { return page * 72; }

// The device arrays and sizes that name a paged cache.
struct Cache {
    uint8_t* data;
    const int* table;  // [n_seqs][max_pages]
    const int* lens;   // [n_seqs]
    long long n_pages;
    int max_pages;
    int page_shift;  // log2(tokens per page)
    int kv_heads;

    __device__ __forceinline__ int page() const { return 1 << page_shift; }
    __device__ __forceinline__ long long block_bytes() const {
        return (long long)kTokenBytes << page_shift;
    }
    // The block of position `pos` of sequence `n`, head `h`; null where the
    // table names no page of the cache.
    __device__ __forceinline__ uint8_t* block(int n, int pos, int h) const {
        const int p = pos >> page_shift;
        if (p >= max_pages) return nullptr;
        const int id = __ldg(table + (long long)n * max_pages + p);
        if (id < 0 || id >= n_pages) return nullptr;
        return data + ((long long)id * kv_heads + h) * block_bytes();
    }
};

}  // namespace attn

// Argument checks shared by the calls on a paged cache (attn_kv4.cu).
kda_status validate_cache(const char* fn, const void* cache, int64_t n_pages, int page,
                          const int* table, int max_pages, const int* lens, int n_seqs,
                          int kv_heads, int head_dim);
// Stride and alignment of a [rows][heads][128] argument (attn_prefill.cu).
kda_status validate_rows(const char* fn, const char* name, const void* p, int64_t stride,
                         int heads);

}  // namespace kda
