// anvil_norm.h -- parameter blocks of the layer-norm kernels (internal to libanvil).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace anvil {

struct NormFwdParams {
    const void* x;        // [rows, width], row stride ldx elements
    const void* weight;   // [width] or null
    const void* bias;     // [width] or null
    void* y;              // [rows, width], row stride ldy
    float* mean;          // [rows] or null
    float* rstd;          // [rows] or null
    long long rows, ldx, ldy;
    int width;
    int dtype, weight_dtype;
    int team_rows;        // rows of a team of the ring kernel (set by the launcher)
    float eps;
    unsigned* err;
};

struct NormBwdParams {
    const void* dy;
    const void* x;
    const float* mean;
    const float* rstd;
    const void* weight;    // or null (1)
    const void* res;       // gradient added to dx, or null
    void* dx;
    float* dweight;        // [width] or null
    float* dbias;          // [width] or null
    float* part;           // [blocks][2][width] partial sums (blocks > 1)
    long long rows, lddy, ldx, ldr, lddx;
    int width;
    int dtype, weight_dtype;
    // set by norm_bwd_plan:
    int blocks;            // of the row pass; 1: it writes dweight and dbias itself
    int vec;               // every array on 16-byte boundaries row by row
    int team_rows;         // rows of a team of the ring kernel (0: the plain kernel)
    unsigned* err;
};

// The most blocks the backward row pass takes for these sizes (whatever the alignment): the
// number of partial rows the workspace holds.
int norm_bwd_max_blocks(long long rows, int width, int dtype);
void norm_bwd_plan(NormBwdParams* p);
cudaError_t launch_norm_fwd(const NormFwdParams& p, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormBwdParams& p, cudaStream_t stream);
cudaError_t launch_norm_grads(const NormBwdParams& p, cudaStream_t stream);

}  // namespace anvil
