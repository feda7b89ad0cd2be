// Scored prefill kernels for block-scaled 8-bit pools, f16 queries.
#include "prefill_launch.cuh"

namespace pagedkv {

cudaError_t prefill_scored_block_f16(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    using namespace pf;
    return launch_block<__half, kModsAny>(pool, c, stream);
}

}  // namespace pagedkv
