// anvil_logprob.h -- parameter blocks of the token log-probability kernels (internal to
// libanvil).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace anvil {

constexpr int LOGPROB_MAX_TOP = 32;  // one list entry per lane of a warp

struct LogprobParams {
    const void* logits;     // [rows, vocab], row stride ld elements
    const void* targets;    // [rows] int32 or int64, or null
    float* logprob;         // [rows] or null (null with targets null)
    float* entropy;         // [rows] or null
    float* lse;             // [rows] or null
    float* top_logprob;     // [rows, top]
    int* top_index;         // [rows, top]
    long long rows, ld;
    int vocab, top;
    int dtype, target64;
};

struct LogprobGradParams {
    const void* logits;
    const void* targets;
    const float* lse;           // [rows]
    const float* entropy;       // [rows], with grad_entropy
    const float* grad_logprob;  // [rows] or null
    const float* grad_entropy;  // [rows] or null
    void* dlogits;              // [rows, vocab], row stride ldd
    long long rows, ld, ldd;
    int vocab;
    int dtype, target64;
};

// Blocks per row of the backward pass.
int logprob_bwd_segments(int vocab, int dtype);
cudaError_t launch_logprob_fwd(const LogprobParams& p, int sm_count, cudaStream_t stream);
cudaError_t launch_logprob_bwd(const LogprobGradParams& p, cudaStream_t stream);

}  // namespace anvil
