// Scored prefill kernels (capped, biased, masked) for 16-bit pools, f16 queries.
#include "prefill_launch.cuh"

namespace pagedkv {

cudaError_t prefill_scored_f16(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    using namespace pf;
    return launch_scored<__half>(pool, c, stream);
}

}  // namespace pagedkv
