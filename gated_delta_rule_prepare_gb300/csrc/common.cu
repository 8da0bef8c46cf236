// Error reporting, status words and the version string of libkda.
#include <mutex>

#include "kda_common.h"

namespace kda {

static thread_local char g_last_error[512] = "";

void set_error(const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
}

bool fault_injected(const char* what) {
    const char* s = getenv("KDA_FAULT_INJECT");
    return s && strcmp(s, what) == 0;
}

// The units' status words, fetched and cleared together: one copy to the host for
// all of them (each word read by a copy of its own: 60 us a call for six,
// and 82 with another copy to clear it).
constexpr int kStatusWords = 9;
struct StatusWords {
    unsigned* at[kStatusWords];
};
__device__ unsigned g_fetched[kStatusWords];
__global__ void fetch_status_kernel(StatusWords words) {
    const int i = threadIdx.x;
    if (i < kStatusWords) g_fetched[i] = atomicExch(words.at[i], 0u);
}

static cudaError_t fetch_status(unsigned (&out)[kStatusWords]) {
    static std::mutex one_at_a_time;  // g_fetched is one for all callers
    std::lock_guard<std::mutex> hold(one_at_a_time);
    cudaError_t (*const where[kStatusWords])(unsigned**) = {
        status_word_prefill, status_word_conv, status_word_prefill_tc,
        status_word_attn,    status_word_kv4,  status_word_decode,
        status_word_pages,   status_word_lin,  status_word_lin_walk};
    StatusWords words;
    for (int i = 0; i < kStatusWords; ++i) {
        const cudaError_t e = where[i](&words.at[i]);
        if (e != cudaSuccess) return e;
    }
    void* args[] = {&words};
    const cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void*>(fetch_status_kernel),
                                           dim3(1), dim3(32), args, 0, nullptr);
    return e != cudaSuccess ? e : cudaMemcpyFromSymbol(out, g_fetched, sizeof(out));
}

}  // namespace kda

extern "C" const char* kda_last_error(void) { return kda::g_last_error; }

extern "C" const char* kda_version(void) { return "libkda 0.1 (sm_103a)"; }

extern "C" kda_status kda_sync_status(uint64_t stream) {
    cudaError_t e = cudaStreamSynchronize(kda::as_stream(stream));
    if (e != cudaSuccess) {
        kda::set_error("kda_sync_status: stream error: %s", cudaGetErrorString(e));
        return KDA_ERR_CUDA;
    }
    unsigned w[kda::kStatusWords];
    e = kda::fetch_status(w);
    if (e != cudaSuccess) {
        kda::set_error("kda_sync_status: reading the status word failed: %s",
                       cudaGetErrorString(e));
        return KDA_ERR_CUDA;
    }
    const unsigned a = w[0] | w[2], b = w[1], d = w[3] | w[4] | w[5] | w[6];
    const unsigned l = w[7] | w[8], all = a | b | d | l;
    if (all) {
        kda::set_error("kda_sync_status: device-side check failed (prefill 0x%x, conv 0x%x, "
                       "attention 0x%x, linear attention 0x%x): %s",
                       a, b, d, l,
                       (all & kda::STATUS_TIMEOUT)      ? "a bounded wait timed out"
                       : (all & kda::STATUS_SMEM_ALIGN) ? "shared memory misaligned"
                       : (all & kda::STATUS_BAD_PAGES)  ? "lens or page_table outside the cache"
                       : (all & kda::STATUS_NO_PAGES)   ? "no free pages left"
                                                        : "malformed cu_seqlens");
        return KDA_ERR_DEVICE;
    }
    return KDA_OK;
}
