// Scored prefill kernels for block-scaled 8-bit pools, bf16 queries.
#include "prefill_launch.cuh"

namespace pagedkv {

cudaError_t prefill_scored_block_bf16(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    using namespace pf;
    return launch_block<__nv_bfloat16, kModsAny>(pool, c, stream);
}

}  // namespace pagedkv
