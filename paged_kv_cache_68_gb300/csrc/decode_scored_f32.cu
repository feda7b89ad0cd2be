// Scored decode kernels (capped, biased, masked) for fp32 pools.
#include "decode_kernel.cuh"

namespace pagedkv {

cudaError_t decode_dispatch_scored_f32(const kv_pool& pool, const DecodeCall& call,
                                   const DecodePlan& plan, cudaStream_t stream) {
    return dec::dispatch<float, true>(pool, call, plan, stream);
}

cudaError_t decode_attrs_scored_f32(const kv_pool& pool, int group, size_t smem, int* ctas_per_sm) {
    return dec::attrs<float, true>(pool, group, smem, ctas_per_sm);
}

}  // namespace pagedkv
