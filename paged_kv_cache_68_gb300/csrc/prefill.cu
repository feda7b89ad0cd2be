// Paged (chunked) prefill: host-side checks and the choice of the kernel's
// translation unit; prefill_launch.cuh launches.
#include <cstdint>

#include "pagedkv_internal.cuh"

namespace pagedkv {

cudaError_t prefill_f16(const kv_pool&, const PrefillCall&, cudaStream_t);
cudaError_t prefill_bf16(const kv_pool&, const PrefillCall&, cudaStream_t);
cudaError_t prefill_block_f16(const kv_pool&, const PrefillCall&, cudaStream_t);
cudaError_t prefill_block_bf16(const kv_pool&, const PrefillCall&, cudaStream_t);
cudaError_t prefill_scored_f16(const kv_pool&, const PrefillCall&, cudaStream_t);
cudaError_t prefill_scored_bf16(const kv_pool&, const PrefillCall&, cudaStream_t);
cudaError_t prefill_scored_q8_f16(const kv_pool&, const PrefillCall&, cudaStream_t);
cudaError_t prefill_scored_q8_bf16(const kv_pool&, const PrefillCall&, cudaStream_t);
cudaError_t prefill_scored_block_f16(const kv_pool&, const PrefillCall&, cudaStream_t);
cudaError_t prefill_scored_block_bf16(const kv_pool&, const PrefillCall&, cudaStream_t);

cudaError_t launch_prefill(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    const bool bf = pool.dtype == KV_BF16;
    if (!bf && pool.dtype != KV_F16) return cudaErrorNotSupported;
    if (pool.block_scales) {
        if (c.mods) return (bf ? prefill_scored_block_bf16 : prefill_scored_block_f16)(pool, c, stream);
        return (bf ? prefill_block_bf16 : prefill_block_f16)(pool, c, stream);
    }
    if (c.mods && is_q8(pool))
        return (bf ? prefill_scored_q8_bf16 : prefill_scored_q8_f16)(pool, c, stream);
    if (c.mods) return (bf ? prefill_scored_bf16 : prefill_scored_f16)(pool, c, stream);
    return (bf ? prefill_bf16 : prefill_f16)(pool, c, stream);
}

}  // namespace pagedkv

static kv_status prefill_impl(kv_pool_t pool, const void* q, void* out, const int32_t* cu_seqlens,
                              int num_tokens, int max_query_len, const int32_t* block_tables,
                              int max_blocks_per_seq, const int32_t* seq_lens, int batch,
                              int num_q_heads, float scale, int num_kv_heads,
                              const kv_score_mods* mods, void* stream, const char* what) {
    if (!pool || batch < 1 || num_q_heads < 1 || num_tokens < 0) return KV_EINVAL;
    if (num_kv_heads != pool->num_kv_heads || num_q_heads % num_kv_heads) return KV_EINVAL;
    const int g = num_q_heads / num_kv_heads;
    if (g != 1 && g != 2 && g != 4 && g != 8) return KV_EUNSUPPORTED;
    if ((pool->dtype != KV_BF16 && pool->dtype != KV_F16) || pool->head_dim != 128 ||
        !pool->has_swizzled_maps)
        return KV_EUNSUPPORTED;
    const int bs = pool->block_size;
    if (bs < 8 || bs > 128 || (bs & (bs - 1))) return KV_EUNSUPPORTED;
    if (pagedkv::is_q8(*pool) && bs < 16) return KV_EUNSUPPORTED;
    if (batch > 65535 || num_kv_heads > 65535) return KV_EUNSUPPORTED;
    if (num_tokens == 0) return KV_OK;
    if (max_query_len < 1 || max_query_len > num_tokens) return KV_EINVAL;
    if (!q || !out || !cu_seqlens || !block_tables || !seq_lens) return KV_EINVAL;
    auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    auto a4 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
    if (!a16(q) || !a16(out) || !a4(cu_seqlens) || !a4(block_tables) || !a4(seq_lens))
        return KV_EINVAL;
    if (max_blocks_per_seq < 1 ||
        (long long)batch * max_blocks_per_seq >= (1ll << 31) ||
        (long long)max_blocks_per_seq * bs >= (1ll << 31))
        return KV_EINVAL;
    if ((long long)num_tokens * num_q_heads * 128 >= (1ll << 40)) return KV_EINVAL;
    if (!(scale > 0.f) || !(scale < 3.4e38f)) return KV_EINVAL;
    pagedkv::PrefillCall call{q,            out,
                              cu_seqlens,   num_tokens,
                              max_query_len, block_tables,
                              max_blocks_per_seq, seq_lens,
                              batch,        num_q_heads,
                              scale,        mods};
    cudaError_t e = pagedkv::launch_prefill(*pool, call, static_cast<cudaStream_t>(stream));
    if (e == cudaErrorNotSupported) return KV_EUNSUPPORTED;
    return e == cudaSuccess ? KV_OK : pagedkv::cuda_fail(e, what);
}

extern "C" {

kv_status paged_attention_prefill(kv_pool_t pool, const void* q, void* out,
                                  const int32_t* cu_seqlens, int num_tokens, int max_query_len,
                                  const int32_t* block_tables, int max_blocks_per_seq,
                                  const int32_t* seq_lens, int batch, int num_q_heads,
                                  float scale, int num_kv_heads, void* stream) {
    const pagedkv::NvtxRange range("paged_attention_prefill");
    return prefill_impl(pool, q, out, cu_seqlens, num_tokens, max_query_len, block_tables,
                        max_blocks_per_seq, seq_lens, batch, num_q_heads, scale, num_kv_heads,
                        nullptr, stream, "paged_attention_prefill");
}

kv_status paged_attention_prefill_scored(kv_pool_t pool, const void* q, void* out,
                                         const int32_t* cu_seqlens, int num_tokens,
                                         int max_query_len, const int32_t* block_tables,
                                         int max_blocks_per_seq, const int32_t* seq_lens,
                                         int batch, int num_q_heads, float scale, int num_kv_heads,
                                         const kv_score_mods* mods, void* stream) {
    const pagedkv::NvtxRange range("paged_attention_prefill_scored");
    if (!pool || !pagedkv::mods_ok(mods)) return KV_EINVAL;
    if (!pagedkv::on_pool_device(*pool)) return KV_EINVAL;
    return prefill_impl(pool, q, out, cu_seqlens, num_tokens, max_query_len, block_tables,
                        max_blocks_per_seq, seq_lens, batch, num_q_heads, scale, num_kv_heads,
                        mods, stream, "paged_attention_prefill_scored");
}

}  // extern "C"
