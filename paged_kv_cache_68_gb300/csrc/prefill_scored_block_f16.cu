// Scored prefill kernels for block-scaled 8-bit pools, f16 queries.
#include "prefill_launch.cuh"

namespace pagedkv {

cudaError_t prefill_scored_block_f16(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    return pf::launch_block<__half, true>(pool, c, stream);
}

}  // namespace pagedkv
