// anvil_multi.cu -- several products in one launch of the pair kernel (PairMultiParams): sums of
// products, two results at once, scaled results.
#include "anvil_linear.cuh"

namespace anvil {

namespace {
template <typename T>
cudaError_t pick(const PairMultiParams& p, int sm_count, cudaStream_t s) {
    return p.box_bytes == 64 ? run_pair<T, 64, MultiPair>(p, sm_count, s) : run_pair<T, 128, MultiPair>(p, sm_count, s);
}
}  // namespace

cudaError_t multi_prepare() {
    cudaError_t e;
#define ANVIL_SMEM(T, W)                                                                                        \
    if ((e = cudaFuncSetAttribute(pair_gemm_kernel<T, W, MultiPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, \
                                  Staging<W>::SMEM)))                                                           \
    return e
    ANVIL_SMEM(__nv_bfloat16, 64);
    ANVIL_SMEM(__nv_bfloat16, 128);
    ANVIL_SMEM(__half, 64);
    ANVIL_SMEM(__half, 128);
    ANVIL_SMEM(float, 64);
    ANVIL_SMEM(float, 128);
#undef ANVIL_SMEM
    return cudaSuccess;
}

cudaError_t launch_pair_multi(const PairMultiParams& p, int sm_count, cudaStream_t s) {
    if (p.epi.out_f32) return pick<float>(p, sm_count, s);
    return p.f16 ? pick<__half>(p, sm_count, s) : pick<__nv_bfloat16>(p, sm_count, s);
}

}  // namespace anvil
