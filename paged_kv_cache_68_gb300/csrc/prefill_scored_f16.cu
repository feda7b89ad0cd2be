// Scored prefill kernels (capped, biased, masked) for 16-bit pools and 8-bit pools
// with pool or token scales, f16 queries.
#include "prefill_launch.cuh"

namespace pagedkv {

cudaError_t prefill_scored_f16(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    return pf::launch_format<__half, true>(pool, c, stream);
}

}  // namespace pagedkv
