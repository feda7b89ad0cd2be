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
// Bound by HBM at 2 bytes read and 1 written per element for prompt chunks, by
// latency for a decode step.  Launches back to back, 8 heads: 256 rows of a
// decode step 5.9 us (1.6 MB), 8191 rows of 17 chunks 16.3 us (50 MB, 3.1 TB/s;
// 20.5 us with the rows out of L2).  What keeps the chunks from the 7.5 us of
// their bytes is each CTA's chain slots -> leader -> notes -> rows -> scale
// -> codes, which the two halves of the batch below overlap in part.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "pagedkv_internal.cuh"

namespace pagedkv {
namespace {

constexpr int kThreads = 256;
constexpr int kD = 128;
constexpr int kMaxRows = 256;             // the largest block size
constexpr int kHeld = 8;                  // row pairs a warp keeps in registers
constexpr int kScanTokens = 1024;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kTiny = 1.17549435e-38f;  // 2^-126

struct BlockAppend {
    const uint4 *fresh_k, *fresh_v;       // the call's K and V rows
    unsigned char *codes_k, *codes_v;
    float *scales_k, *scales_v;
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

// The bits above which a 16-bit value's magnitude is an infinity or NaN.
template <typename T> constexpr uint32_t kInfBits = 0x7c00u;
template <> constexpr uint32_t kInfBits<__nv_bfloat16> = 0x7f80u;

// Q of four values, one word.  INT8: rounded to nearest even by the addition of
// 1.5 * 2^23, whose sum holds the integer in its low byte (an FMA-pipe step; a
// conversion instruction takes the MUFU's pipe, at an eighth of the rate; the
// packed addition is not used: the compiler fused it with the product before it,
// which must be rounded first).  No clamp: |x| (1 / new) is at most
// 127 (1 + 2^-22), and a factor below 1 only shrinks a code, so every sum rounds
// within [-127, 127].
template <bool INT8> __device__ __forceinline__ uint32_t encode4(float2 a, float2 b) {
    if constexpr (INT8) {
        auto bits = [](float y) { return __float_as_uint(__fadd_rn(y, 12582912.f)); };
        return __byte_perm(__byte_perm(bits(a.x), bits(a.y), 0x0040),
                           __byte_perm(bits(b.x), bits(b.y), 0x0040), 0x5410);
    } else {
        return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
               ((uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16);
    }
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
    const float2 f2 = make_float2(f, f);
    return encode4<INT8>(__fmul2_rn(make_float2(v[0], v[1]), f2),
                         __fmul2_rn(make_float2(v[2], v[3]), f2));
}

__global__ void __launch_bounds__(kThreads) mark_rows_kernel(const BlockAppend p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long ii = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (ii >= p.num_tokens) return;
    const int i = (int)ii;
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
    float* scale = (part ? p.scales_v : p.scales_k) + (size_t)blk * p.hkv + h;
    const float old = tok[0] != 0 ? 0.f : *scale;
    unsigned char* base = (part ? p.codes_v : p.codes_k) + ((size_t)blk * p.bs * p.hkv + h) * kD;
    const uint4* fresh = (part ? p.fresh_v : p.fresh_k) + (size_t)h * (kD / 8) + hl;
    const size_t row_bytes = (size_t)p.hkv * kD, fresh_row = (size_t)p.hkv * (kD / 8);
    uint4 w[kHeld];
    auto load = [&](int g) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int n = g + 2 * k + half;
            w[k] = make_uint4(0u, 0u, 0u, 0u);
            if (n < nw) w[k] = __ldg(fresh + (size_t)(tok[rows[n]] - 1) * fresh_row);
        }
    };
    // The largest magnitude, as 16-bit patterns: without their sign they order as
    // the values do, two to an instruction.
    uint32_t top = 0u;
#pragma unroll 1
    for (int g = 0; g < nw; g += 2 * kHeld) {
        load(g);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            top = __vmaxu2(top, __vmaxu2(w[k].x & 0x7fff7fffu, w[k].y & 0x7fff7fffu));
            top = __vmaxu2(top, __vmaxu2(w[k].z & 0x7fff7fffu, w[k].w & 0x7fff7fffu));
        }
    }
    top = max(top & 0xffffu, top >> 16);
    top = __reduce_max_sync(kAll, top);
    const bool finite = top < kInfBits<T>;
    if (!finite) {                                   // the largest of the finite ones
        top = 0u;
        for (int g = 0; g < nw; g += 2 * kHeld) {
            load(g);
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                const uint32_t ws[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = ws[i] & 0x7fffu, hi = (ws[i] >> 16) & 0x7fffu;
                    top = max(top, max(lo < kInfBits<T> ? lo : 0u, hi < kInfBits<T> ? hi : 0u));
                }
            }
        }
        top = __reduce_max_sync(kAll, top);
    }
    const float a = widen<T>(top).x;
    float now = fmaxf(old, __fdiv_rn(a, INT8 ? 127.f : 448.f));
    if (now < kTiny) now = 0.f;
    if (INT8 && (!finite || old != old)) now = __int_as_float(0x7fc00000);
    // the block's other rows, when the scale grew
    if (nw < p.bs && old > 0.f && now > old) {
        const float f = __fdiv_rn(old, now);
#pragma unroll 1
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
#pragma unroll 1
    for (int g = 0; g < nw; g += 2 * kHeld) {
        if (nw > 2 * kHeld) load(g);                 // (else still held)
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int n = g + 2 * k + half;
            const float2 i2 = make_float2(inv, inv);
            const float2 f0 = __fmul2_rn(widen<T>(w[k].x), i2), f1 = __fmul2_rn(widen<T>(w[k].y), i2);
            const float2 f2 = __fmul2_rn(widen<T>(w[k].z), i2), f3 = __fmul2_rn(widen<T>(w[k].w), i2);
            const uint2 c = make_uint2(encode4<INT8>(f0, f1), encode4<INT8>(f2, f3));
            if (n < nw)
                *reinterpret_cast<uint2*>(base + rows[n] * row_bytes + hl * 8) =
                    INT8 && now != now ? make_uint2(0u, 0u) : c;
        }
    }
    if (lane == 0) *scale = now;
}

// The rows that `tok` has, in order, by one warp: how many.
__device__ __forceinline__ int list_rows(const BlockAppend& p, const int* tok, unsigned char* rows,
                                         int lane) {
    int n = 0;
    for (int r0 = 0; r0 < p.bs; r0 += 32) {
        const bool has = r0 + lane < p.bs && tok[r0 + lane] != 0;
        const unsigned m = __ballot_sync(kAll, has);
        if (has) rows[n + __popc(m & ((1u << lane) - 1u))] = (unsigned char)(r0 + lane);
        n += __popc(m);
    }
    return n;
}

// Up to kScanTokens rows: a CTA per token, which reads all slots itself.
template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads) append_scan_kernel(const BlockAppend p) {
    __shared__ int tok[kMaxRows];
    __shared__ unsigned char rows[kMaxRows];
    __shared__ int nw_s;
    constexpr int kPer = kScanTokens / kThreads;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, i = blockIdx.x;
    const long long slot = p.slots[i];
    long long others[kPer];                          // (in flight with the token's own)
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int j = tid + k * kThreads;
        others[k] = j < p.num_tokens ? p.slots[j] : -1;
    }
    if (tid < p.bs) tok[tid] = 0;
    if (slot < 0) return;                            // padding
    if (slot >= p.num_rows) {
        if (tid == 0) atomicOr(p.err, KV_DEVERR_SLOT_RANGE);
        return;
    }
    const int blk = (int)slot / p.bs;
    const long long first = (long long)blk * p.bs;
    __syncthreads();
    bool later = false;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const long long r = others[k] - first;
        if (others[k] >= 0 && r >= 0 && r < p.bs) {
            const int j = tid + k * kThreads;
            atomicMax(&tok[r], j + 1);
            later = later || j > i;
        }
    }
    if (__syncthreads_or(later)) return;             // a later token leads
    const int warp = tid >> 5, lane = tid & 31;
    if (warp == 0) {
        const int n = list_rows(p, tok, rows, lane);
        if (lane == 0) nw_s = n;
    }
    __syncthreads();
    for (int item = warp; item < 2 * p.hkv; item += kThreads / 32)
        quantise_head<T, INT8>(p, item & 1, item >> 1, blk, tok, rows, nw_s, lane);
}

// Any number, after mark_rows_kernel: a CTA per `chunk` tokens writes the blocks
// that they lead.  The chunk's leaders are found at once, one token a thread, and
// up to kTogether of their blocks are worked on together: a chunk where one
// request's rows end and the next one's begin leads two, and taking them in turn
// made those CTAs last twice as long as the others (36 k cycles of 42 k, while the
// SMs were busy 22 k on average).
constexpr int kTogether = 4;
template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads, 4) append_marked_kernel(const BlockAppend p) {
    __shared__ int tok[kTogether][kMaxRows];
    __shared__ unsigned char rows[kTogether][kMaxRows];
    __shared__ int led[kThreads];
    __shared__ int nw_s[kTogether], led_n;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long i = (long long)blockIdx.x * p.chunk + tid;
    if (tid == 0) led_n = 0;
    __syncthreads();
    if (tid < p.chunk && i < p.num_tokens) {
        const long long slot = p.slots[i];
        if (slot >= 0 && slot < p.num_rows) {
            const int blk = (int)slot / p.bs;
            if (p.leader[blk] == i + 1) {
                p.leader[blk] = 0;                   // (no other token equals it)
                led[atomicAdd(&led_n, 1)] = blk;
            }
        }
    }
    __syncthreads();
    for (int k0 = 0; k0 < led_n; k0 += kTogether) {
        const int nk = min(kTogether, led_n - k0);
        for (int x = tid; x < nk * p.bs; x += kThreads) {
            const int k = x / p.bs, r = x - k * p.bs;
            int* owner = p.owner + (size_t)led[k0 + k] * p.bs + r;
            tok[k][r] = *owner;
            *owner = 0;
        }
        __syncthreads();
        if (warp < nk) {
            const int n = list_rows(p, tok[warp], rows[warp], lane);
            if (lane == 0) nw_s[warp] = n;
        }
        __syncthreads();
        for (int item = warp; item < nk * 2 * p.hkv; item += kThreads / 32) {
            const int k = item / (2 * p.hkv), h = item - k * 2 * p.hkv;
            quantise_head<T, INT8>(p, h & 1, h >> 1, led[k0 + k], tok[k], rows[k], nw_s[k], lane);
        }
        __syncthreads();                             // tok and rows before the next blocks'
    }
}

template <typename T, bool INT8>
cudaError_t launch(const BlockAppend& call, cudaStream_t stream) {
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
        cfg.gridDim = dim3((unsigned)p.num_tokens);
        return cudaLaunchKernelEx(&cfg, append_scan_kernel<T, INT8>, p);
    }
    cfg.gridDim = dim3((unsigned)((p.num_tokens + kThreads - 1) / kThreads));
    cudaError_t e = cudaLaunchKernelEx(&cfg, mark_rows_kernel, p);
    if (e != cudaSuccess) return e;
    // as many tokens to a CTA as fill a block, when they come in order: then most
    // CTAs lead one
    p.chunk = std::min(p.bs, kThreads);
    cfg.gridDim = dim3((unsigned)((p.num_tokens + p.chunk - 1) / p.chunk));
    return cudaLaunchKernelEx(&cfg, append_marked_kernel<T, INT8>, p);
}

}  // namespace

cudaError_t launch_append_block_scaled(const kv_pool& pool, const void* k_new, const void* v_new,
                                       const int64_t* slots, int num_tokens, cudaStream_t stream) {
    if (num_tokens <= 0) return cudaSuccess;
    BlockAppend p = {};
    p.fresh_k = static_cast<const uint4*>(k_new);
    p.fresh_v = static_cast<const uint4*>(v_new);
    p.codes_k = static_cast<unsigned char*>(pool.k);
    p.codes_v = static_cast<unsigned char*>(pool.v);
    p.scales_k = pool.k_scales;
    p.scales_v = pool.v_scales;
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
        return bf ? launch<__nv_bfloat16, true>(p, stream) : launch<__half, true>(p, stream);
    return bf ? launch<__nv_bfloat16, false>(p, stream) : launch<__half, false>(p, stream);
}

}  // namespace pagedkv
