// Rotary positions of the rows that the attention calls take (kda_attn_rope).
// Pair p of a head turns by positions[r][axis of p] * inv_freq[p].
//
// Bound by memory, 512 bytes a row and head.  A CTA takes a few rows: their angles
// first, shared by all heads, then heads in 16-byte pieces.
//
// Angles.  A turn is 2^64: F = inv_freq / (2 pi) in that unit (one FP64 product a pair
// and CTA), and position * F in integers drops whole turns exactly.  F's 53 bits leave
// an angle exact to 2^-53 |position * inv_freq|, below 2^-20 of a turn for all int32 positions
// and frequencies up to 4; sincospif takes the rest.
//
// 69001 rows of 40 heads, three axes (1.4 GB): 208 us, 6.8 TB/s, what a copy takes (in
// halves 209 to 223; halves that are no multiple of 8: 350).  64 rows: 2.6 us, as a call 5.3.
#include "attn_common.h"
#include "f32x2.h"

namespace kda {
namespace {

using namespace attn;

constexpr int kThreads = 256;
constexpr int kMaxPairs = D / 2;

struct RopeArgs {
    const uint16_t* in[2];  // q, k
    uint16_t* out[2];
    long long in_stride[2], out_stride[2];
    int heads[2];
    long long rows;
    const int* positions;
    const float* inv_freq;
    int axes, pairs;
    uint32_t axis[4];  // of each pair, two bits
    float factor;
};

// a, b turned by the pair's angle.
__device__ __forceinline__ float2 turn(float a, float b, float2 cs) {
    return make_float2(fmaf(a, cs.x, -b * cs.y), fmaf(b, cs.x, a * cs.y));
}

// A head's 16-byte piece u (channels 8u..8u+7) with whole pairs next to each other.
template <bool F16>
__device__ __forceinline__ uint4 turn_piece(uint4 x, const float2* cs, int u, int pairs) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = 4 * u + i;
        if (p < pairs) {
            const float2 v = widen2<F16>(w[i]), y = turn(v.x, v.y, cs[p]);
            w[i] = narrow2<F16>(y.x, y.y);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Piece u with the first channels of pairs 8u..8u+7, and the piece with their second ones.
template <bool F16>
__device__ __forceinline__ void turn_pieces(uint4& x, uint4& y, const float2* cs, int u) {
    uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 p = widen2<F16>(xs[e]), w = widen2<F16>(ys[e]);
        const float2 lo = turn(p.x, w.x, cs[8 * u + 2 * e]);
        const float2 hi = turn(p.y, w.y, cs[8 * u + 2 * e + 1]);
        xs[e] = narrow2<F16>(lo.x, hi.x);
        ys[e] = narrow2<F16>(lo.y, hi.y);
    }
    x = make_uint4(xs[0], xs[1], xs[2], xs[3]);
    y = make_uint4(ys[0], ys[1], ys[2], ys[3]);
}
enum Layout { kInterleaved, kHalves8, kHalves };  // kHalves8: pairs a multiple of 8

// Eight threads a head, two 16-byte pieces each: one of first channels of pairs with that
// of the second ones, pieces behind the pairs by twos; interleaved, any two.  (Sixteen with a
// piece each, interleaved, as many loads in flight: 244 us for 69001 rows where this took 211.)
// Or (kHalves) a warp a head, 8 bytes a lane, whose partners come from shared memory.  Threads step through a
// tile's rows and heads, kBatch of them in flight (one more or less: up to a tenth longer).
// An output in its input's place is written behind its reads: a thread's, or a warp's.
constexpr int kRowsTile = 8;  // at most
template <bool F16, int LAYOUT>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a, int tile) {
    __shared__ float2 cs[kRowsTile][kMaxPairs];
    __shared__ unsigned long long unit[kMaxPairs];
    pdl_wait();
    pdl_release();
    const int tid = threadIdx.x;
    if (tid < a.pairs) {
        // the fraction of a turn a position adds, in units of 2^-64 turns
        const double f = (double)__ldg(a.inv_freq + tid) * 0.15915494309189535;
        const double whole = f - floor(f);
        unit[tid] = (unsigned long long)(whole * 18446744073709551616.0);
    }
    const long long row0 = (long long)blockIdx.x * tile;
    const int rows = (int)min((long long)tile, a.rows - row0);
    __syncthreads();
    for (int i = tid; i < rows * kMaxPairs; i += kThreads) {
        const int r = i / kMaxPairs, p = i % kMaxPairs;
        if (p >= a.pairs) continue;
        const uint32_t word = p < 32 ? (p < 16 ? a.axis[0] : a.axis[1])
                                     : (p < 48 ? a.axis[2] : a.axis[3]);
        const int axis = word >> (2 * (p & 15)) & 3;
        const long long pos = __ldg(a.positions + (row0 + r) * a.axes + axis);
        const unsigned long long at = (unsigned long long)pos * unit[p];
        float s, c;
        sincospif((float)((int)(at >> 32)) * 0x1p-31f, &s, &c);
        cs[r][p] = make_float2(c * a.factor, s * a.factor);
    }
    __syncthreads();
    constexpr int LANES = LAYOUT == kHalves ? 32 : 8;
    constexpr int kHeads = kThreads / LANES;  // heads at a time
    constexpr int kBatch = LAYOUT == kHalves ? 2 : 3;
    const int u = tid % LANES, turned = a.pairs / 8;
    __shared__ __align__(16) uint16_t head[LAYOUT == kHalves ? kThreads / 32 : 1][kBatch][D];
    int first = u, second = u + 8;  // of its pieces
    if (LAYOUT == kHalves8) {
        second = u + turned;
        if (u >= turned) first = 2 * u, second = 2 * u + 1;
    }
    const int heads = a.heads[0] + a.heads[1];
    // slots of a tile: heads innermost
    const int total = rows * heads;
    int r = 0, h = tid / LANES;  // of the next slot
    while (h >= heads && r < rows) h -= heads, ++r;
    for (int i0 = tid / LANES; i0 < total; i0 += kBatch * kHeads) {
        const uint16_t* src[kBatch];
        uint16_t* dst[kBatch];
        int row[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            row[k] = r < rows ? r : -1;
            if (r >= rows) continue;
            const bool key = h >= a.heads[0];
            const int head = key ? h - a.heads[0] : h;
            src[k] = (key ? a.in[1] : a.in[0]) +
                     (row0 + r) * (key ? a.in_stride[1] : a.in_stride[0]) + head * D;
            dst[k] = (key ? a.out[1] : a.out[0]) +
                     (row0 + r) * (key ? a.out_stride[1] : a.out_stride[0]) + head * D;
            for (h += kHeads; h >= heads && r < rows; ++r) h -= heads;
        }
        if constexpr (LAYOUT == kHalves) {  // (the same rows and heads for all of a warp)
            uint2 x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (row[k] >= 0) x[k] = reinterpret_cast<const uint2*>(src[k])[u];
            __syncwarp();  // the last heads' partners are read
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (row[k] >= 0) *reinterpret_cast<uint2*>(head[tid >> 5][k] + 4 * u) = x[k];
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (row[k] < 0) continue;
                const float2 lo = widen2<F16>(x[k].x), hi = widen2<F16>(x[k].y);
                float y[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = 4 * u + e;
                    if (c >= 2 * a.pairs) continue;
                    const bool is_first = c < a.pairs;
                    const int p = is_first ? c : c - a.pairs;
                    const float2 t = cs[row[k]][p];
                    const float other =
                        widen2<F16>(head[tid >> 5][k][is_first ? c + a.pairs : p]).x;
                    y[e] = turn(y[e], other, make_float2(t.x, is_first ? t.y : -t.y)).x;
                }
                // (channels behind the pairs as they came: rounding changes NaN)
                uint2 out = x[k];
                if (4 * u < 2 * a.pairs) out.x = narrow2<F16>(y[0], y[1]);
                if (4 * u + 2 < 2 * a.pairs) out.y = narrow2<F16>(y[2], y[3]);
                reinterpret_cast<uint2*>(dst[k])[u] = out;
            }
        } else {
            uint4 x[kBatch], y[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (row[k] < 0) continue;
                x[k] = reinterpret_cast<const uint4*>(src[k])[first];
                y[k] = reinterpret_cast<const uint4*>(src[k])[second];
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (row[k] < 0) continue;
                if (LAYOUT == kInterleaved) {
                    x[k] = turn_piece<F16>(x[k], cs[row[k]], first, a.pairs);
                    y[k] = turn_piece<F16>(y[k], cs[row[k]], second, a.pairs);
                } else if (u < turned) {
                    turn_pieces<F16>(x[k], y[k], cs[row[k]], u);
                }
                reinterpret_cast<uint4*>(dst[k])[first] = x[k];
                reinterpret_cast<uint4*>(dst[k])[second] = y[k];
            }
        }
    }
}

// Rows a CTA: one for each multiprocessor while that makes tiles of a few rows (40 heads: 150 rows
// in tiles of 1 take 2.6 us, of 8 6.5; 1200 rows in tiles of 4 6.4, of 1 8.2), then tiles that
// share their frequencies (69001 rows in tiles of 8 208 us, of 2 236, of 16 211).
int tile_rows(long long rows) {
    return rows <= 152 ? 1 : rows <= 2 * 152 ? 2 : rows <= 8 * 152 ? 4 : kRowsTile;
}

template <bool F16>
void launch_rope(const RopeArgs& a, bool interleaved, dim3 grid, int tile, cudaStream_t s) {
    auto kernel = interleaved        ? rope_kernel<F16, kInterleaved>
                  : a.pairs % 8 == 0 ? rope_kernel<F16, kHalves8>
                                     : rope_kernel<F16, kHalves>;
    launch_pdl(kernel, grid, dim3(kThreads), 0, s, a, tile);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_attn_rope(const void* q, const void* k, void* q_out, void* k_out,
                                    int64_t rows, int heads, int kv_heads, int head_dim,
                                    int in_dtype, int64_t q_row_stride, int64_t k_row_stride,
                                    int64_t q_out_row_stride, int64_t k_out_row_stride,
                                    const int* positions, int axes, const float* inv_freq,
                                    int pairs, const uint8_t* pair_axis, int interleaved,
                                    float factor, uint64_t stream) {
    const char* fn = "kda_attn_rope";
    KDA_REQUIRE(head_dim == D, KDA_ERR_UNSUPPORTED, "%s: head_dim %d unsupported (only 128)", fn,
                head_dim);
    KDA_REQUIRE(in_dtype == KDA_F32 || in_dtype == KDA_BF16 || in_dtype == KDA_F16,
                KDA_ERR_INVALID_ARG, "%s: in_dtype %d is not a kda_dtype", fn, in_dtype);
    KDA_REQUIRE(in_dtype != KDA_F32, KDA_ERR_UNSUPPORTED, "%s: FP32 rows are not built", fn);
    KDA_REQUIRE(rows >= 0 && rows < 0x7fffffffLL && heads >= 1 && kv_heads >= 0 &&
                    (long long)heads + kv_heads <= 1 << 16,
                KDA_ERR_INVALID_ARG,
                "%s: rows (%lld), heads (%d) and kv_heads (%d): 0 to 2^31 - 2 rows, at least one "
                "head, at most 2^16 heads",
                fn, (long long)rows, heads, kv_heads);
    KDA_REQUIRE(axes >= 1 && axes <= 4, KDA_ERR_INVALID_ARG, "%s: axes (%d) must be 1 to 4", fn,
                axes);
    KDA_REQUIRE(pairs >= 1 && pairs <= kMaxPairs, KDA_ERR_INVALID_ARG,
                "%s: pairs (%d) must be 1 to %d", fn, pairs, kMaxPairs);
    KDA_REQUIRE(isfinite(factor), KDA_ERR_INVALID_ARG, "%s: factor must be finite", fn);
    RopeArgs a = {};
    for (int p = 0; pair_axis && p < pairs; ++p) {
        KDA_REQUIRE(pair_axis[p] < axes, KDA_ERR_INVALID_ARG, "%s: pair %d has axis %d of %d", fn,
                    p, pair_axis[p], axes);
        a.axis[p >> 4] |= (uint32_t)pair_axis[p] << (2 * (p & 15));
    }
    if (rows == 0) return KDA_OK;
    kda_status st = validate_rows(fn, "q", q, q_row_stride, heads);
    if (st == KDA_OK) st = validate_rows(fn, "q_out", q_out, q_out_row_stride, heads);
    if (st == KDA_OK && kv_heads) st = validate_rows(fn, "k", k, k_row_stride, kv_heads);
    if (st == KDA_OK && kv_heads)
        st = validate_rows(fn, "k_out", k_out, k_out_row_stride, kv_heads);
    if (st != KDA_OK) return st;
    KDA_REQUIRE((q != q_out || q_row_stride == q_out_row_stride) &&
                    (!kv_heads || k != k_out || k_row_stride == k_out_row_stride),
                KDA_ERR_INVALID_ARG, "%s: an output in its input's place has its row stride", fn);
    KDA_REQUIRE(positions && inv_freq, KDA_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    KDA_REQUIRE((reinterpret_cast<uintptr_t>(positions) & 3) == 0 &&
                    (reinterpret_cast<uintptr_t>(inv_freq) & 3) == 0,
                KDA_ERR_INVALID_ARG, "%s: positions and inv_freq must be 4-byte aligned", fn);
    KDA_REQUIRE(!fault_injected(), KDA_ERR_CUDA, "%s: injected launch failure", fn);
    a.in[0] = (const uint16_t*)q;
    a.in[1] = (const uint16_t*)k;
    a.out[0] = (uint16_t*)q_out;
    a.out[1] = (uint16_t*)k_out;
    a.in_stride[0] = q_row_stride, a.in_stride[1] = k_row_stride;
    a.out_stride[0] = q_out_row_stride, a.out_stride[1] = k_out_row_stride;
    a.heads[0] = heads, a.heads[1] = kv_heads;
    a.rows = rows, a.positions = positions, a.inv_freq = inv_freq;
    a.axes = axes, a.pairs = pairs, a.factor = factor;
    const int tile = tile_rows(rows);
    const dim3 grid((unsigned)((rows + tile - 1) / tile));
    if (in_dtype == KDA_F16) launch_rope<true>(a, interleaved, grid, tile, as_stream(stream));
    else launch_rope<false>(a, interleaved, grid, tile, as_stream(stream));
    return launch_result(fn);
}
