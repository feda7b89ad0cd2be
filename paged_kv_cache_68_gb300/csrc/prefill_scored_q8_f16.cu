// Scored prefill kernels for 8-bit pools with pool or token scales, f16 queries.
#include "prefill_launch.cuh"

namespace pagedkv {

cudaError_t prefill_scored_q8_f16(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    using namespace pf;
    return launch_q8<__half, kModsAny>(pool, c, stream);
}

}  // namespace pagedkv
