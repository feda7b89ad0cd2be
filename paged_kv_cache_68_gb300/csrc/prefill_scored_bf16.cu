// Scored prefill kernels (capped, biased, masked) for 16-bit pools, bf16 queries.
#include "prefill_launch.cuh"

namespace pagedkv {

cudaError_t prefill_scored_bf16(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    using namespace pf;
    return launch_scored<__nv_bfloat16>(pool, c, stream);
}

}  // namespace pagedkv
