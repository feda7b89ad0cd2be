// A step's bookkeeping on the GPU: block tables, slot mapping, positions,
// query offsets and lengths, from the requests' lengths alone.
//
// What is computed ("Part 3: single node" (random-liu.github.io), ch. 13
// sec. 1: the batch's new tokens are flattened into one stream with request
// boundaries, and slot = table[pos / bs] * bs + pos % bs; "Lecture 3"
// (semidirectx.com, CS349D notes), sec. 3.1: a block is taken from the free
// list only when the last one is full).  With old_b = ceil(ctx_b / bs) and
// need_b = ceil((ctx_b + new_b) / bs) - old_b:
//   cu_b  = sum of new_c over c < b,   off_b = head + sum of need_c over c < b,
//   table[b][old_b + k] = free[off_b + k]   (k < need_b),
//   token i of request b: position p = ctx_b + i, slot as above.
//
// Every block that a request gains holds at least one of its new tokens, and
// the block's first row is one of them (p % bs == 0, p >= ctx_b), so the token
// at a block's first row enters the block in the table: the tokens cover the
// table's new entries exactly once, and no pass over the tables is needed.
//
// One launch.  Each CTA scans all requests itself (two block-wide sums, in
// shared memory; at most 4096 requests, 32 KB) and then places its own
// contiguous share of the tokens: a redundant scan out of L2 costs less than
// a second launch and needs no workspace.  Bound by latency: the chain lengths
// -> sums -> free id or table entry -> slot.  Launches back to back: 256 decoding
// requests (13 KB) 3.8 us, 1000 prompts of 403,000 tokens (5.1 MB, 0.8 us of HBM
// time) 7.1 us.
#include <algorithm>

#include "pagedkv_internal.cuh"

namespace pagedkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanPer = kMaxBatch / kPlanThreads;   // requests per thread, at most

struct PlanParams {
    const int32_t* ctx;
    const int32_t* fresh;            // new tokens of each request
    int32_t* tables;
    const int32_t* free_blocks;
    const int32_t* head;
    int32_t* head_out;
    int32_t* cu;
    int32_t* lens;
    int64_t* slots;
    int32_t* positions;              // may be null
    int* err;
    int batch, max_blocks, num_free, num_tokens, num_blocks, bs;
};

// Exclusive sum of one long long per thread over the CTA (every thread calls).
__device__ __forceinline__ long long excl_sum(long long v, long long* scratch, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long long w = scratch[lane];
        const long long own = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        scratch[lane] = w - own;
        if (lane == 31) scratch[32] = w;
    }
    __syncthreads();
    const long long r = scratch[warp] + x - v;
    *total = scratch[32];
    __syncthreads();                 // scratch is read before its next use
    return r;
}

__global__ void __launch_bounds__(kPlanThreads) plan_step_kernel(const PlanParams p) {
    __shared__ int cu_s[kMaxBatch + 1];
    __shared__ int off_s[kMaxBatch];         // first free-list index; -1: not placed
    __shared__ long long scratch[kPlanWarps + 1];
    __shared__ int last_s;                   // end of the handed-out part of the free list
    static_assert(kPlanWarps == 32, "the sums' second level is one warp");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int tid = threadIdx.x, B = p.batch, bs = p.bs;
    const bool first_cta = blockIdx.x == 0;
    const long long cap = (long long)p.max_blocks * bs;
    const int head_raw = *p.head;
    const int head = min(max(head_raw, 0), p.num_free);
    int err = head != head_raw ? KV_DEVERR_BLOCK_RANGE : 0;
    if (tid == 0) last_s = head;

    // -- 1. the requests: offsets of their tokens, then of their blocks ---------
    const int per = (B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(B, tid * per), n = min(B, b0 + per) - b0;
    int ctx[kPlanPer], add[kPlanPer];
    long long sum = 0;
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
        ctx[k] = add[k] = 0;
        if (k < n) {
            ctx[k] = p.ctx[b0 + k];
            add[k] = p.fresh[b0 + k];
        }
    }
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
        if (ctx[k] < 0 || add[k] < 0) {
            err |= KV_DEVERR_SEQ_RANGE;
            ctx[k] = max(ctx[k], 0);
            add[k] = 0;
        }
        sum += add[k];
    }
    long long total;
    long long run = excl_sum(sum, scratch, &total);
    const long long T = p.num_tokens;
    long long need[kPlanPer];
    bool fits[kPlanPer];
    sum = 0;
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
        need[k] = 0;
        fits[k] = false;
        if (k < n) {
            cu_s[b0 + k] = (int)min(run, T);
            run += add[k];
            const long long end = (long long)ctx[k] + add[k];
            if (end > cap) err |= KV_DEVERR_SEQ_RANGE;
            else if (run > T) err |= KV_DEVERR_QUERY_RANGE;
            else {
                fits[k] = true;
                need[k] = (end + bs - 1) / bs - (ctx[k] + (long long)bs - 1) / bs;
            }
            sum += need[k];
        }
    }
    if (tid == 0) cu_s[B] = (int)min(total, T);
    long long taken;
    run = head + excl_sum(sum, scratch, &taken);
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k)
        if (k < n) {
            bool placed = fits[k];
            if (need[k] > 0 && run + need[k] > p.num_free) {
                placed = false;
                err |= KV_DEVERR_NO_BLOCKS;
            }
            off_s[b0 + k] = placed ? (int)run : -1;
            if (placed && need[k] > 0) atomicMax(&last_s, (int)(run + need[k]));
            run += need[k];
            if (first_cta) p.lens[b0 + k] = ctx[k] + (placed ? add[k] : 0);
        }
    if (err && first_cta) atomicOr(p.err, err);
    __syncthreads();
    if (first_cta) {
        for (int b = tid; b <= B; b += kPlanThreads) p.cu[b] = cu_s[b];
        if (tid == 0) *p.head_out = last_s;
    }

    // -- 2. this CTA's share of the tokens -----------------------------------------
    const int share = (int)(((long long)p.num_tokens + gridDim.x - 1) / gridDim.x);
    const int i1 = (int)min((long long)p.num_tokens, (long long)(blockIdx.x + 1) * share);
    const int live = cu_s[B];
    for (long long ii = (long long)blockIdx.x * share + tid; ii < i1; ii += kPlanThreads) {
        const int i = (int)ii;
        long long slot = -1;
        int pos = 0;
        if (i < live) {
            // the last request with cu <= i (one with no tokens shares its
            // successor's offset, so it is never the last)
            int lo = 0, hi = B;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu_s[mid] <= i) lo = mid; else hi = mid;
            }
            const int c = max(p.ctx[lo], 0);
            pos = (int)min((long long)c + (i - cu_s[lo]), 0x7fffffffll);
            const int off = off_s[lo];
            if (off >= 0) {
                const int j = pos / bs, r = pos - j * bs;
                const int old = c / bs + (c % bs != 0);
                int32_t* entry = p.tables + (size_t)lo * p.max_blocks + j;
                const int id = j >= old ? p.free_blocks[off + j - old] : *entry;
                if (j >= old && r == 0) *entry = id;
                if (id >= 0 && id < p.num_blocks) slot = (long long)id * bs + r;
                else atomicOr(p.err, KV_DEVERR_BLOCK_RANGE);
            }
        }
        p.slots[i] = slot;
        if (p.positions) p.positions[i] = pos;
    }
}

}  // namespace
}  // namespace pagedkv

extern "C" kv_status kv_plan_step(kv_pool_t pool, const int32_t* context_lens,
                                  const int32_t* new_lens, int batch, int32_t* block_tables,
                                  int max_blocks_per_seq, const int32_t* free_blocks, int num_free,
                                  const int32_t* free_head, int32_t* free_head_out,
                                  int32_t* cu_seqlens, int32_t* seq_lens, int64_t* slot_mapping,
                                  int32_t* positions, int num_tokens, void* stream) {
    const pagedkv::NvtxRange range("kv_plan_step");
    if (!pool || batch < 1 || num_tokens < 0 || num_free < 0 || max_blocks_per_seq < 1)
        return KV_EINVAL;
    if (batch > pagedkv::kMaxBatch) return KV_EUNSUPPORTED;
    if (!context_lens || !new_lens || !block_tables || !free_head || !free_head_out ||
        !cu_seqlens || !seq_lens || (num_free > 0 && !free_blocks) ||
        (num_tokens > 0 && !slot_mapping))
        return KV_EINVAL;
    const void* p4[] = {context_lens, new_lens, block_tables, free_blocks, free_head,
                        free_head_out, cu_seqlens, seq_lens, positions};
    for (const void* p : p4)
        if (reinterpret_cast<uintptr_t>(p) & 3u) return KV_EINVAL;
    if (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) return KV_EINVAL;
    // every CTA reads the inputs while one writes the results: none may be both
    if (free_head == free_head_out || context_lens == seq_lens || new_lens == seq_lens)
        return KV_EINVAL;
    if ((long long)max_blocks_per_seq * pool->block_size >= (1ll << 31)) return KV_EINVAL;
    if (!pagedkv::on_pool_device(*pool)) return KV_EINVAL;
    pagedkv::PlanParams p;
    p.ctx = context_lens;
    p.fresh = new_lens;
    p.tables = block_tables;
    p.free_blocks = free_blocks;
    p.head = free_head;
    p.head_out = free_head_out;
    p.cu = cu_seqlens;
    p.lens = seq_lens;
    p.slots = slot_mapping;
    p.positions = positions;
    p.err = pool->d_err;
    p.batch = batch;
    p.max_blocks = max_blocks_per_seq;
    p.num_free = num_free;
    p.num_tokens = num_tokens;
    p.num_blocks = pool->num_blocks;
    p.bs = pool->block_size;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max(1, std::min(pool->num_sms,
                                                      (int)(((long long)num_tokens + pagedkv::kPlanThreads - 1) /
                                                            pagedkv::kPlanThreads))));
    cfg.blockDim = dim3(pagedkv::kPlanThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, pagedkv::plan_step_kernel, p);
    return e == cudaSuccess ? KV_OK : pagedkv::cuda_fail(e, "kv_plan_step");
}
