// anvil_adamw.h -- parameter blocks and launchers of the AdamW kernels (internal to libanvil).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace anvil {

constexpr int ADAMW_BLOCK = 256;           // consecutive values that share a scale
constexpr int ADAMW_FEW = 16, ADAMW_MANY = 448;  // tensors of a launch (the parameter block takes 32 KB at most)

// param's storage: fp32, bf16, fp16, or bf16 with the fp32 value's low half beside it
enum : int { ADAMW_F32 = 0, ADAMW_BF16 = 1, ADAMW_F16 = 2, ADAMW_SPLIT = 3 };

struct AdamwTensor {
    void* p;
    uint16_t* low;   // ADAMW_SPLIT
    const void* g;
    void* m;         // fp32, or e4m3 codes
    void* v;         // fp32, or codes of the root
    float* scales;   // [2][blocks] of the codes
    long long count;
    int chunk0;      // the launch's chunks before this tensor's
};
template <int N>
struct AdamwParams {
    AdamwTensor t[N];
    int tensors;
    int chunk;               // blocks of a thread block's chunk
    float beta1, c1, beta2, c2, eps;
    float scalars[4];        // step_size, root, decay, grad_scale
    const float* d_scalars;  // or null: the same on the device
};
struct AdamwGroup {
    AdamwParams<ADAMW_MANY> p;
    int chunks;
};
// Blocks of 256 values of a thread block's chunk: one to four turns of its eight warps, as many as still
// leave every SM eight chunks.  (3M bf16 values with 8-bit states and their decoding, us, on vector
// boundaries and off them: 16 and 22 in chunks of 8 or 16, 22 and 26 of 32; 50M split bf16 values 190 of 32,
// 193 of 64.)
inline int adamw_chunk(long long blocks) {
    int chunk = 8;
    while (chunk < 32 && blocks >= 152ll * 8 * chunk) chunk *= 2;
    return chunk;
}

// param: ADAMW_*, grad: DT_*, vec: every array on the boundaries of four values
cudaError_t launch_adamw(const AdamwGroup& g, int param, int grad, bool codes, bool vec, cudaStream_t s);

// What codes stand for: m = code scale, v = (root code scale)^2, written to p and g's place as
// fp32 (AdamwTensor.p = m's values, .low unused, .g = v's).
cudaError_t launch_adamw_values(const AdamwGroup& g, bool vec, cudaStream_t s);

}  // namespace anvil
