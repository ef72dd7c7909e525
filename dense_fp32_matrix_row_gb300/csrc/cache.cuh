// cache.cuh -- shared parts of the attention operators over an 8-bit paged
// key-value cache: argument structs and launchers.
#pragma once

#include "q8.cuh"
#include "sgemm_gb300.h"

namespace sgemm_gb300 {

// Bit of the error word: an index that a kernel read from device memory lies outside its array.
constexpr unsigned kErrBadIndex = 2u;

// Heads whose keys and values the operators take: multiples of 16 elements.
constexpr int64_t kCacheMaxDim = 256;

// Attention takes its scores in base 2: a scale times this has to be finite.
constexpr float kLog2e = 1.44269504088896341f;

struct HeadRowsArgs {
    int64_t T;
    int D, type;
    sgemm_heads q, q_out, k, k_out, v;    // .p == nullptr: not there
    const float *q_weight, *k_weight;     // or nullptr
    float eps;
    sgemm_rotary rotary;                  // dims == 0: none
    const int64_t *slots;                 // with `cache`
    sgemm_q8_cache cache;                 // .k == nullptr: none
    cudaStream_t stream;
    unsigned *err;
    int sm_count;
};

struct CacheReadArgs {
    int64_t N;
    int type;
    sgemm_q8_cache cache;
    const int64_t *slots;
    sgemm_heads k_out, v_out;             // .p == nullptr: not wanted
    cudaStream_t stream;
    unsigned *err;
    int sm_count;
};

struct AttendArgs {
    int B, Hk, G, D, type;
    sgemm_heads q, out;
    sgemm_q8_cache cache;
    const int32_t *table;
    int64_t ld_table;
    int width;                            // columns of the table
    const int32_t *lens;
    float scale;
    int window;                           // 0: the whole sequence
    float *lse;                           // or nullptr
    cudaStream_t stream;
    unsigned *err;
    int sm_count;
};

cudaError_t launch_head_rows(const HeadRowsArgs &a);
cudaError_t launch_cache_read(const CacheReadArgs &a);
// Bytes of partial results that a call may write.
size_t attend_workspace_bytes(const AttendArgs &a);
#ifdef __CUDACC__
// Launches `kernel` as a programmatic dependent of the work before it: its blocks may
// be set up while that finishes, and wait (pdl_wait) before they touch memory.
template <typename Params>
cudaError_t launch_dependent(void (*kernel)(Params), unsigned blocks, unsigned threads, size_t smem, cudaStream_t stream,
                             const Params &params) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, params);
}
#endif
// `tickets`: kAttendTickets words that are zero, and zero again once the call has run.
constexpr int kAttendTickets = 4096;
cudaError_t launch_attend(const AttendArgs &a, void *workspace, unsigned *tickets);

}  // namespace sgemm_gb300
