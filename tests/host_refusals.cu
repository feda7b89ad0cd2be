// Host argument checks of the calls that need a pool, on a pool description made
// here without a device: every refusal answers before anything touches the GPU.
// Prints "ok" or the first call that answered otherwise; exit status 0 / 1.
#include <cstdio>
#include <limits>

#include "pagedkv_internal.cuh"

static int failures = 0;
static void expect(kv_status got, kv_status want, const char* what) {
    if (got != want) {
        std::printf("%s: %d, not %d\n", what, (int)got, (int)want);
        ++failures;
    }
}

int main() {
    kv_pool pool;
    pool.num_blocks = 8;
    pool.block_size = 16;
    pool.num_kv_heads = 2;
    pool.head_dim = 128;
    pool.dtype = pool.cache_dtype = KV_BF16;
    pool.elem_bytes = 2;
    pool.has_swizzled_maps = true;
    pool.device = 0;
    pool.num_sms = 152;
    pool.d_err = nullptr;
    alignas(16) static char mem[4096];
    auto* i32 = reinterpret_cast<int32_t*>(mem);
    auto* i64 = reinterpret_cast<int64_t*>(mem);
    const float nan = std::numeric_limits<float>::quiet_NaN(), inf = std::numeric_limits<float>::infinity();

    auto plan = [&](int batch, int width, int free_n, int tokens, int32_t* head_out, int32_t* lens,
                    const int32_t* ctx, int64_t* slots) {
        return kv_plan_step(&pool, ctx, i32 + 8, batch, i32 + 16, width, i32 + 24, free_n, i32 + 32, head_out,
                            i32 + 48, lens, slots, nullptr, tokens, nullptr);
    };
    expect(plan(0, 4, 4, 1, i32 + 40, i32 + 56, i32, i64 + 40), KV_EINVAL, "batch 0");
    expect(plan(4097, 4, 4, 1, i32 + 40, i32 + 56, i32, i64 + 40), KV_EUNSUPPORTED, "batch 4097");
    expect(plan(1, 0, 4, 1, i32 + 40, i32 + 56, i32, i64 + 40), KV_EINVAL, "no table width");
    expect(plan(1, 1 << 28, 4, 1, i32 + 40, i32 + 56, i32, i64 + 40), KV_EINVAL, "2^32 positions");
    expect(plan(1, 4, -1, 1, i32 + 40, i32 + 56, i32, i64 + 40), KV_EINVAL, "free list of -1");
    expect(plan(1, 4, 4, -1, i32 + 40, i32 + 56, i32, i64 + 40), KV_EINVAL, "-1 tokens");
    expect(plan(1, 4, 4, 1, i32 + 32, i32 + 56, i32, i64 + 40), KV_EINVAL, "head in place");
    expect(plan(1, 4, 4, 1, i32 + 40, i32, i32, i64 + 40), KV_EINVAL, "lengths in place");
    expect(plan(1, 4, 4, 1, i32 + 40, i32 + 56, i32, nullptr), KV_EINVAL, "no slots");
    expect(plan(1, 4, 4, 1, i32 + 40, i32 + 56, nullptr, i64 + 40), KV_EINVAL, "no lengths");
    expect(plan(1, 4, 4, 1, i32 + 40, i32 + 56, reinterpret_cast<int32_t*>(mem + 2), i64 + 40), KV_EINVAL,
           "misaligned lengths");

    auto dec = [&](const kv_score_mods* m, int width) {
        return paged_attention_decode_scored(&pool, mem, mem, i32, width, i32, 1, 4, 0.1f, 2, m, mem, 16,
                                             nullptr);
    };
    auto pre = [&](const kv_score_mods* m) {
        return paged_attention_prefill_scored(&pool, mem, mem, i32, 1, 1, i32, 4, i32, 1, 4, 0.1f, 2, m,
                                              nullptr);
    };
    expect(dec(nullptr, 4), KV_EINVAL, "decode without mods");
    expect(pre(nullptr), KV_EINVAL, "prefill without mods");
    for (float cap : {-1.f, nan, inf, 1e9f, 1e-9f, 1025.f}) {
        kv_score_mods m = {};
        m.softcap = cap;
        expect(dec(&m, 4), KV_EINVAL, "decode with a cap out of range");
        expect(pre(&m), KV_EINVAL, "prefill with a cap out of range");
    }
    kv_score_mods m = {};
    m.window = -1;
    expect(dec(&m, 4), KV_EINVAL, "decode, window -1");
    expect(pre(&m), KV_EINVAL, "prefill, window -1");
    m = {};
    m.alibi_slopes = reinterpret_cast<const float*>(mem + 1);
    expect(dec(&m, 4), KV_EINVAL, "decode, misaligned slopes");
    m = {};
    m.first_visible = reinterpret_cast<const int32_t*>(mem + 2);
    expect(pre(&m), KV_EINVAL, "prefill, misaligned first_visible");
    m = {};
    m.prefix_lens = i32;
    expect(dec(&m, 4), KV_EINVAL, "decode with a prefix");
    m = {};
    expect(dec(&m, 1 << 28), KV_EINVAL, "decode, 2^32 positions");
    std::printf("%s\n", failures ? "failed" : "ok");
    return failures != 0;
}
