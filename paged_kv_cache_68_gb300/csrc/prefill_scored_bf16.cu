// Scored prefill kernels (capped, biased, masked) for 16-bit pools and 8-bit pools
// with pool or token scales, bf16 queries.
#include "prefill_launch.cuh"

namespace pagedkv {

cudaError_t prefill_scored_bf16(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    return pf::launch_format<__nv_bfloat16, true>(pool, c, stream);
}

}  // namespace pagedkv
