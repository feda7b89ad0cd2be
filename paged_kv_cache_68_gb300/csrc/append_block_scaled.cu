// kv_append on a block-scaled 8-bit pool: one scale for each (block, KV head).
//
// The rows that one call writes into a block share its scales, so they are
// handled together: for K and V and every head, a = max |x| over the rows,
//   new = max(old, a / qmax),  code = Q(x * (1 / new)),
// and, when the scale grew, the block's other rows are rounded again by
// old / new (pagedkv.h states the arithmetic step by step).  ("Part 3: single
// node" (random-liu.github.io), ch. 10 sec. 1 and 3: K and V are scaled and
// rounded to 8 bits when written, with a scale for a group of values.)
//
// The token with the highest index of a block's rows leads: its CTA writes the
// whole block, a warp per (head, K or V); a row repeated in the call is the
// highest index's.  Which rows a block gets is found in one of two ways:
//   SCAN, up to kScanTokens rows: every CTA reads the call's slots and keeps
//     those of its block (one launch; a 1024-slot scan is 8 KB out of L2);
//   otherwise a first kernel notes each row's index at its slot and each
//     block's highest index with atomic maxima, and the leaders read their
//     block's notes and clear them (4 bytes a slot; any order of slots).
// Bound by HBM at 2 bytes read and 1 written per element for prompt chunks,
// by latency for a decode step.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "pagedkv_internal.cuh"

namespace pagedkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kD = 128;
constexpr int kMaxRows = 256;             // the largest block size
constexpr int kHeld = 8;                  // row pairs a warp keeps in registers
constexpr int kScanTokens = 1024;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kTiny = 1.17549435e-38f;  // 2^-126

struct BlockAppend {
    const uint4* fresh[2];                // the call's K and V rows
    unsigned char* codes[2];
    float* scales[2];
    const int64_t* slots;
    int* owner;
    int* leader;
    int* err;
    long long num_rows;
    int num_tokens, bs, hkv, chunk;
};

template <typename T> __device__ __forceinline__ float2 widen(uint32_t w);
template <> __device__ __forceinline__ float2 widen<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <> __device__ __forceinline__ float2 widen<__nv_bfloat16>(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

__device__ __forceinline__ uint32_t int8_code(float y) {
    return (uint32_t)min(127, max(-127, __float2int_rn(y))) & 0xffu;
}

// Q of two values: the low 16 bits hold their codes.
template <bool INT8> __device__ __forceinline__ uint32_t encode2(float a, float b) {
    if constexpr (INT8) return int8_code(a) | (int8_code(b) << 8);
    else return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Four codes, each rounded again after a factor.
template <bool INT8> __device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
    float v[4];
    if constexpr (INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)(int)(signed char)((w >> (8 * i)) & 0xffu);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)((w >> (16 * i)) & 0xffffu), __NV_E4M3);
            const float2 x = __half22float2(__half2(h));
            v[2 * i] = x.x;
            v[2 * i + 1] = x.y;
        }
    }
    return encode2<INT8>(__fmul_rn(v[0], f), __fmul_rn(v[1], f)) |
           (encode2<INT8>(__fmul_rn(v[2], f), __fmul_rn(v[3], f)) << 16);
}

__global__ void __launch_bounds__(kThreads) mark_rows_kernel(const BlockAppend p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= p.num_tokens) return;
    const long long slot = p.slots[i];
    if (slot < 0) return;
    if (slot >= p.num_rows) {
        atomicOr(p.err, KV_DEVERR_SLOT_RANGE);
        return;
    }
    atomicMax(p.owner + slot, i + 1);
    atomicMax(p.leader + (int)slot / p.bs, i + 1);
}

// One (head, K or V) of a block, by one warp: the rows in tok (row -> index of
// its token + 1, 0: not written), listed in rows[0 .. nw).  Half a warp holds a
// row's 128 values, 8 a lane.
template <typename T, bool INT8>
__device__ __forceinline__ void quantise_head(const BlockAppend& p, int part, int h, int blk,
                                              const int* tok, const unsigned char* rows, int nw,
                                              int lane) {
    const int half = lane >> 4, hl = lane & 15;
    float* scale = p.scales[part] + (size_t)blk * p.hkv + h;
    const float old = tok[0] != 0 ? 0.f : *scale;
    unsigned char* base = p.codes[part] + ((size_t)blk * p.bs * p.hkv + h) * kD;
    const size_t row_bytes = (size_t)p.hkv * kD;
    uint4 w[kHeld];
    auto load = [&](int g) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int n = g + 2 * k + half;
            w[k] = make_uint4(0u, 0u, 0u, 0u);
            if (n < nw)
                w[k] = __ldg(p.fresh[part] +
                             ((size_t)(tok[rows[n]] - 1) * p.hkv + h) * (kD / 8) + hl);
        }
    };
    float a = 0.f;
    bool finite = true;
    for (int g = 0; g < nw; g += 2 * kHeld) {
        load(g);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const uint32_t ws[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = widen<T>(ws[i]);
                const bool fx = isfinite(f.x), fy = isfinite(f.y);
                a = fmaxf(a, fmaxf(fx ? fabsf(f.x) : 0.f, fy ? fabsf(f.y) : 0.f));
                finite = finite && fx && fy;
            }
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kAll, a, o));
    finite = __all_sync(kAll, finite);
    float now = fmaxf(old, __fdiv_rn(a, INT8 ? 127.f : 448.f));
    if (now < kTiny) now = 0.f;
    if (INT8 && (!finite || old != old)) now = __int_as_float(0x7fc00000);
    // the block's other rows, when the scale grew
    if (nw < p.bs && old > 0.f && now > old) {
        const float f = __fdiv_rn(old, now);
        for (int r = lane >> 3; r < p.bs; r += 4)
            if (tok[r] == 0) {
                uint4* c = reinterpret_cast<uint4*>(base + r * row_bytes) + (lane & 7);
                uint4 v = *c;
                v.x = rescale4<INT8>(v.x, f);
                v.y = rescale4<INT8>(v.y, f);
                v.z = rescale4<INT8>(v.z, f);
                v.w = rescale4<INT8>(v.w, f);
                *c = v;
            }
    }
    const float inv = now > 0.f ? __fdiv_rn(1.f, now) : 0.f;   // (0 for a NaN scale)
    for (int g = 0; g < nw; g += 2 * kHeld) {
        if (nw > 2 * kHeld) load(g);                 // (else still held)
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int n = g + 2 * k + half;
            const uint32_t ws[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = widen<T>(ws[i]);
                c[i] = encode2<INT8>(__fmul_rn(f.x, inv), __fmul_rn(f.y, inv));
            }
            if (n < nw)
                *reinterpret_cast<uint2*>(base + rows[n] * row_bytes + hl * 8) =
                    INT8 && now != now ? make_uint2(0u, 0u)
                                       : make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        }
    }
    if (lane == 0) *scale = now;
}

template <typename T, bool INT8, bool SCAN>
__global__ void __launch_bounds__(kThreads) append_block_kernel(const BlockAppend p) {
    __shared__ int tok[kMaxRows];
    __shared__ unsigned char rows[kMaxRows];
    __shared__ int nw_s;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int i0 = blockIdx.x * p.chunk, i1 = min(p.num_tokens, i0 + p.chunk);
    for (int i = i0; i < i1; ++i) {                  // (every branch below is CTA-uniform)
        const long long slot = p.slots[i];
        if (slot < 0) continue;                      // padding
        if (slot >= p.num_rows) {
            if (SCAN && tid == 0) atomicOr(p.err, KV_DEVERR_SLOT_RANGE);
            continue;
        }
        const int blk = (int)slot / p.bs;
        if constexpr (SCAN) {
            const long long first = (long long)blk * p.bs;
            if (tid < p.bs) tok[tid] = 0;
            __syncthreads();
            bool later = false;
            for (int j = tid; j < p.num_tokens; j += kThreads) {
                const long long r = p.slots[j] - first;
                if (r >= 0 && r < p.bs) {
                    atomicMax(&tok[r], j + 1);
                    later = later || j > i;
                }
            }
            if (__syncthreads_or(later)) continue;   // a later token leads
        } else {
            if (p.leader[blk] != i + 1) continue;
            if (tid < p.bs) {
                tok[tid] = p.owner[(size_t)blk * p.bs + tid];
                p.owner[(size_t)blk * p.bs + tid] = 0;
            }
            __syncthreads();                         // every thread has read the leader
            if (tid == 0) p.leader[blk] = 0;
        }
        if (warp == 0) {
            int n = 0;
            for (int r0 = 0; r0 < p.bs; r0 += 32) {
                const bool has = r0 + lane < p.bs && tok[r0 + lane] != 0;
                const unsigned m = __ballot_sync(kAll, has);
                if (has) rows[n + __popc(m & ((1u << lane) - 1u))] = (unsigned char)(r0 + lane);
                n += __popc(m);
            }
            if (lane == 0) nw_s = n;
        }
        __syncthreads();
        const int nw = nw_s;
        for (int item = warp; item < 2 * p.hkv; item += kWarps)
            quantise_head<T, INT8>(p, item & 1, item >> 1, blk, tok, rows, nw, lane);
        __syncthreads();                             // tok and rows before the next token's
    }
}

template <typename T, bool INT8>
cudaError_t launch(const kv_pool& pool, const BlockAppend& call, cudaStream_t stream) {
    BlockAppend p = call;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (p.num_tokens <= kScanTokens) {
        p.chunk = 1;
        cfg.gridDim = dim3((unsigned)p.num_tokens);
        return cudaLaunchKernelEx(&cfg, append_block_kernel<T, INT8, true>, p);
    }
    cfg.gridDim = dim3((unsigned)((p.num_tokens + kThreads - 1) / kThreads));
    cudaError_t e = cudaLaunchKernelEx(&cfg, mark_rows_kernel, p);
    if (e != cudaSuccess) return e;
    // about four CTAs' worth of tokens per SM: most tokens lead no block
    p.chunk = std::max(1, p.num_tokens / (4 * pool.num_sms));
    cfg.gridDim = dim3((unsigned)((p.num_tokens + p.chunk - 1) / p.chunk));
    return cudaLaunchKernelEx(&cfg, append_block_kernel<T, INT8, false>, p);
}

}  // namespace

cudaError_t launch_append_block_scaled(const kv_pool& pool, const void* k_new, const void* v_new,
                                       const int64_t* slots, int num_tokens, cudaStream_t stream) {
    if (num_tokens <= 0) return cudaSuccess;
    BlockAppend p = {};
    p.fresh[0] = static_cast<const uint4*>(k_new);
    p.fresh[1] = static_cast<const uint4*>(v_new);
    p.codes[0] = static_cast<unsigned char*>(pool.k);
    p.codes[1] = static_cast<unsigned char*>(pool.v);
    p.scales[0] = pool.k_scales;
    p.scales[1] = pool.v_scales;
    p.slots = slots;
    p.owner = pool.d_owner;
    p.leader = pool.d_leader;
    p.err = pool.d_err;
    p.num_rows = (long long)pool.num_blocks * pool.block_size;
    p.num_tokens = num_tokens;
    p.bs = pool.block_size;
    p.hkv = pool.num_kv_heads;
    const bool bf = pool.dtype == KV_BF16;
    if (pool.cache_dtype == KV_INT8)
        return bf ? launch<__nv_bfloat16, true>(pool, p, stream) : launch<__half, true>(pool, p, stream);
    return bf ? launch<__nv_bfloat16, false>(pool, p, stream) : launch<__half, false>(pool, p, stream);
}

}  // namespace pagedkv
