// Scored prefill kernels for 8-bit pools with pool or token scales, bf16 queries.
#include "prefill_launch.cuh"

namespace pagedkv {

cudaError_t prefill_scored_q8_bf16(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    using namespace pf;
    return launch_q8<__nv_bfloat16, kModsAny>(pool, c, stream);
}

}  // namespace pagedkv
