// Decode kernels for block-scaled 8-bit pools with bf16 queries and outputs.
#include "decode_kernel.cuh"

namespace pagedkv {

cudaError_t decode_dispatch_block_bf16(const kv_pool& pool, const DecodeCall& call,
                                   const DecodePlan& plan, cudaStream_t stream) {
    return dec::dispatch_q8<__nv_bfloat16, dec::kScBlock>(pool, call, plan, stream);
}

cudaError_t decode_attrs_block_bf16(const kv_pool& pool, int group, size_t smem, int* ctas_per_sm) {
    return dec::attrs_q8<__nv_bfloat16, dec::kScBlock>(pool, group, smem, ctas_per_sm);
}

}  // namespace pagedkv
