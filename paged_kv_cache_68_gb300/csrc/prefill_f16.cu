// Prefill kernels for 16-bit pools and 8-bit pools with pool or token scales, f16 queries.
#include "prefill_launch.cuh"

namespace pagedkv {

cudaError_t prefill_f16(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    using namespace pf;
    return launch_plain<__half>(pool, c, stream);
}

}  // namespace pagedkv
