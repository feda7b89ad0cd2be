// Paged (chunked) prefill: the per-call query tensor map and the launch of the
// tcgen05 kernel (prefill_kernel.cuh), for the translation units that
// instantiate it (one per query type and kind of kernel).
#pragma once

#include <cstdint>

#include "prefill_kernel.cuh"

namespace pagedkv {
namespace pf {

// FMT: -1 for 16-bit pools, else the 8-bit pool's code format; SC: its kind of
// scales; MODS: scored prefill's kind.
template <typename T, int G, int FMT, int SC, int MODS>
cudaError_t launch_typed(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    constexpr bool Q8 = FMT >= 0;
    constexpr int QT = BM / G;
    // q viewed as [T rows][Hq][D]; one box = QT rows x the group's G heads x
    // 64 dims (128 bytes, swizzled), so the tile lands as row = query * G + head
    CUtensorMap tmap_q;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)c.num_q_heads,
                                (cuuint64_t)c.num_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2u, (cuuint64_t)c.num_q_heads * D * 2u};
    const cuuint32_t box[3] = {64u, (cuuint32_t)G, (cuuint32_t)QT};
    if (!encode_tiled_map(&tmap_q, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(c.q), dims,
                          strides, box, true))
        return cudaErrorInvalidValue;
    // K/V boxes of min(bs, BN) rows: the pool's swizzled maps (box = one
    // block; 8-bit pools: 128 code bytes = all dims) when a block fits a KV
    // tile, else maps with BN-row boxes
    const CUtensorMap* mk = &pool.tmap_k_swz;
    const CUtensorMap* mv = &pool.tmap_v_swz;
    CUtensorMap tk, tv;
    if (pool.block_size > BN) {
        const cuuint64_t elt = Q8 ? 1u : 2u;
        const cuuint64_t kdims[3] = {(cuuint64_t)D, (cuuint64_t)pool.num_kv_heads,
                                     (cuuint64_t)pool.num_blocks * (cuuint64_t)pool.block_size};
        const cuuint64_t kstr[2] = {(cuuint64_t)D * elt, (cuuint64_t)pool.num_kv_heads * D * elt};
        const cuuint32_t kbox[3] = {Q8 ? 128u : 64u, 1u, (cuuint32_t)BN};
        const CUtensorMapDataType dt = Q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
        if (!encode_tiled_map(&tk, dt, 3, pool.k, kdims, kstr, kbox, true) ||
            !encode_tiled_map(&tv, dt, 3, pool.v, kdims, kstr, kbox, true))
            return cudaErrorInvalidValue;
        mk = &tk;
        mv = &tv;
    }
    auto kern = paged_prefill<T, G, FMT, SC, MODS>;
    constexpr uint32_t smem_bytes = Lay<Q8>::bytes;
    cudaError_t e = dec::allow_smem<paged_prefill<T, G, FMT, SC, MODS>>(pool.device, smem_bytes);
    if (e != cudaSuccess) return e;
    Params p;
    p.q = c.q;
    p.out = c.out;
    p.cu_seqlens = c.cu_seqlens;
    p.block_tables = c.block_tables;
    p.seq_lens = c.seq_lens;
    p.err = pool.d_err;
    p.num_tokens = c.num_tokens;
    p.max_blocks = c.max_blocks;
    p.batch = c.batch;
    p.num_q_heads = c.num_q_heads;
    p.num_blocks = pool.num_blocks;
    p.bs = pool.block_size;
    p.max_q = c.max_query_len;
    p.box_rows = pool.block_size < BN ? pool.block_size : BN;
    // FP8: the K scale multiplies every score, the V scale the output
    const bool fp8 = pool.cache_dtype == KV_FP8_E4M3;
    p.qscale = c.scale * 1.4426950408889634f * (fp8 ? pool.fp8_k_scale : 1.f);
    p.vscale = fp8 ? pool.fp8_v_scale : 1.f;
    p.k_scales = pool.k_scales;
    p.v_scales = pool.v_scales;
    p.num_kv_heads = pool.num_kv_heads;
    p.wait_ns = pool.wait_ns;
    p.softcap = c.mods ? c.mods->softcap : 0.f;
    p.inv_softcap = p.softcap > 0.f ? 1.f / p.softcap : 0.f;
    p.slopes = c.mods ? c.mods->alibi_slopes : nullptr;
    p.window = c.mods ? c.mods->window : 0;
    p.first = c.mods ? c.mods->first_visible : nullptr;
    p.prefix = c.mods ? c.mods->prefix_lens : nullptr;
    cudaLaunchConfig_t cfg = {};
    // one CTA per pair of query tiles
    cfg.gridDim = dim3((unsigned)((c.max_query_len + 2 * QT - 1) / (2 * QT)),
                       (unsigned)pool.num_kv_heads, (unsigned)c.batch);
    cfg.blockDim = dim3(FMT >= 0 ? NTHREADS_Q8 : NTHREADS);
    cfg.dynamicSmemBytes = smem_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tmap_q, *mk, *mv, p);
}

template <typename T, int FMT, int SC, int MODS>
cudaError_t launch_group(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    switch (c.num_q_heads / pool.num_kv_heads) {
        case 1: return launch_typed<T, 1, FMT, SC, MODS>(pool, c, stream);
        case 2: return launch_typed<T, 2, FMT, SC, MODS>(pool, c, stream);
        case 4: return launch_typed<T, 4, FMT, SC, MODS>(pool, c, stream);
        case 8: return launch_typed<T, 8, FMT, SC, MODS>(pool, c, stream);
    }
    return cudaErrorNotSupported;
}

// 8-bit pools with pool or token scales; MODS: 0 or kModsAny.
template <typename T, int MODS>
cudaError_t launch_q8(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    if (pool.cache_dtype == KV_FP8_E4M3)
        return launch_group<T, dec::kFmtE4M3, dec::kScPool, MODS>(pool, c, stream);
    return launch_group<T, dec::kFmtInt8, dec::kScToken, MODS>(pool, c, stream);
}

// Block-scaled pools.
template <typename T, int MODS>
cudaError_t launch_block(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    if (pool.cache_dtype == KV_FP8_E4M3)
        return launch_group<T, dec::kFmtE4M3, dec::kScBlock, MODS>(pool, c, stream);
    return launch_group<T, dec::kFmtInt8, dec::kScBlock, MODS>(pool, c, stream);
}

// Plain prefill of 16-bit and 8-bit pools.
template <typename T>
cudaError_t launch_plain(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    if (is_q8(pool)) return launch_q8<T, 0>(pool, c, stream);
    return launch_group<T, -1, dec::kScPool, 0>(pool, c, stream);
}

// Scored prefill of 16-bit pools: the kernel of the call's kind.
template <typename T>
cudaError_t launch_scored(const kv_pool& pool, const PrefillCall& c, cudaStream_t stream) {
    constexpr int m = kModsMask, sc = dec::kScPool;
    const bool cap = c.mods->softcap > 0.f, bias = c.mods->alibi_slopes != nullptr;
    if (cap && bias) return launch_group<T, -1, sc, m | kModsCap | kModsBias>(pool, c, stream);
    if (cap) return launch_group<T, -1, sc, m | kModsCap>(pool, c, stream);
    if (bias) return launch_group<T, -1, sc, m | kModsBias>(pool, c, stream);
    return launch_group<T, -1, sc, m>(pool, c, stream);
}

}  // namespace pf
}  // namespace pagedkv
