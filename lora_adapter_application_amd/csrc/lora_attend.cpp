// lora_attend.cpp -- the C ABI of what stands between a layer's projections, declared in
// include/lora_mi355x.h: head norms with rotary positions (lora_norm_rotary_group), the paged
// cache (lora_cache_*) and attention over it (lora_attend_*).
//
// A cache is device memory of its ctx, cut in pages whose order and lengths the caller keeps; its
// calls read and write what their arguments name and keep nothing else.  The attention's plans and
// parts live in a workspace of the ctx that grows with the batches prepared; memory that a
// captured graph may use stays allocated until lora_slots_destroy.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/lora_mi355x.h"
#include "lora_attend.h"
#include "lora_ctx.h"

using namespace lora;

namespace {

constexpr int32_t kMostHeads = 1024;

bool overlap(const void *p, size_t pb, const void *q, size_t qb)
{
    return (uintptr_t)p < (uintptr_t)q + qb && (uintptr_t)q < (uintptr_t)p + pb;
}

int before_launch(lora_ctx *c, hipStream_t s)
{
    StreamState *st = stream_state(c, s);
    if (!st)
        return fail(c, LORA_ERR_HIP, "hipEventCreateWithFlags failed");
    st->since_fence = true;
    return LORA_OK;
}

int check_tokens(lora_ctx *c, int32_t n_tokens)
{
    if (n_tokens < 0)
        return fail(c, LORA_ERR_INVALID_ARGUMENT, "n_tokens %d < 0", n_tokens);
    if (n_tokens > c->max_tokens)
        return fail(c, LORA_ERR_TOO_MANY_TOKENS, "n_tokens %d > max_tokens %d", n_tokens, c->max_tokens);
    return LORA_OK;
}

int check_cache(lora_ctx *c, const lora_cache *cache)
{
    for (const auto &p : c->caches)
        if (p.get() == cache)
            return LORA_OK;
    return fail(c, LORA_ERR_INVALID_ARGUMENT, "not a cache of this ctx");
}

bool any_capture(const lora_ctx *c, hipStream_t s)
{
    if (s && stream_capturing(s))
        return true;
    for (const auto &st : c->streams)
        if (st.stream && stream_capturing(st.stream))
            return true;
    return false;
}

// The capture that s is part of, or 0.
unsigned long long capture_of(hipStream_t s)
{
    if (!s)
        return 0;
    hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (hipStreamGetCaptureInfo(s, &status, &id) != hipSuccess) {
        (void)hipGetLastError();
        return 0;
    }
    return status == hipStreamCaptureStatusNone ? 0 : id;
}

int device_alloc(lora_ctx *c, void **p, size_t bytes, const char *what)
{
    c->allocations.reserve(c->allocations.size() + 1);
    const hipError_t e = hipMalloc(p, bytes);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        *p = nullptr;
        return fail(c, (e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation) ? LORA_ERR_OUT_OF_MEMORY
                                                                                  : LORA_ERR_HIP,
                    "%s (%zu bytes): %s", what, bytes, hipGetErrorString(e));
    }
    c->allocations.push_back(*p);
    return LORA_OK;
}

// The host containers may throw: nothing leaves a C entry but a status.
template <typename F>
int guarded(F &&f) noexcept
{
    try {
        return f();
    } catch (const std::bad_alloc &) {
        return LORA_ERR_OUT_OF_MEMORY;
    } catch (...) {
        return LORA_ERR_HIP;
    }
}

int do_norm_rotary(lora_ctx *ctx, const lora_rotary *rotary, int32_t n, const int32_t *modules,
                   const void *const *x, const void *const *weight, double eps, void *const *y,
                   const int32_t *positions, int32_t n_tokens, void *stream)
{
    if (check_ctx(ctx))
        return LORA_ERR_INVALID_ARGUMENT;
    ctx->last_error.clear();
    int rc = check_group(ctx, n, modules);
    if (rc || (rc = check_tokens(ctx, n_tokens)))
        return rc;
    if (!rotary || rotary->head_dim < 2 || rotary->head_dim % 2 || rotary->rotary_dim < 2 ||
        rotary->rotary_dim % 2 || rotary->rotary_dim > rotary->head_dim ||
        rotary->rotary_dim > LORA_ROTARY_MAX_DIM ||
        (rotary->layout != LORA_ROTARY_HALF && rotary->layout != LORA_ROTARY_INTERLEAVED))
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "rotary is not what lora_rotary_init forms");
    if (rotary->head_dim > LORA_NORM_MAX_DIM)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "head_dim %d exceeds LORA_NORM_MAX_DIM", rotary->head_dim);
    if (!(eps >= 0.0) || !std::isfinite((float)eps))
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
    for (int i = 0; i < n; ++i)
        if (ctx->shapes[modules[i]].d_out % rotary->head_dim)
            return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "module %d: d_out %d is not whole heads of %d",
                        modules[i], ctx->shapes[modules[i]].d_out, rotary->head_dim);
    if (n_tokens == 0)
        return LORA_OK;
    if (!positions)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "positions is NULL");
    if ((rc = check_ptrs(ctx, n, x, "x", false)) ||
        (rc = check_ptrs(ctx, n, (const void *const *)y, "y", true)))
        return rc;
    NormArgs a;
    std::memset(&a, 0, sizeof a);
    a.rot.rot = *rotary;
    a.rot.n = n;
    a.rot.T = n_tokens;
    a.rot.positions = positions;
    a.eps = (float)eps;
    const int V = 16 / ctx->elem;
    bool vec = rotary->head_dim % V == 0 && rotary->rotary_dim % V == 0 &&
               (rotary->layout == LORA_ROTARY_INTERLEAVED || rotary->rotary_dim / 2 % V == 0);
    for (int i = 0; i < n; ++i) {
        const int d_out = ctx->shapes[modules[i]].d_out;
        const size_t bytes = (size_t)n_tokens * d_out * ctx->elem;
        for (int j = 0; j < n; ++j) {
            const size_t other = (size_t)n_tokens * ctx->shapes[modules[j]].d_out * ctx->elem;
            if ((!(i == j && x[j] == y[i]) && overlap(y[i], bytes, x[j], other)) ||
                (i != j && overlap(y[i], bytes, y[j], other)))
                return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "y[%d] overlaps x or y of member %d", i, j);
            if (weight && weight[j] && overlap(y[i], bytes, weight[j], (size_t)rotary->head_dim * ctx->elem))
                return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "y[%d] overlaps the weight of member %d", i, j);
        }
        if (overlap(y[i], bytes, positions, sizeof(int32_t) * (size_t)n_tokens))
            return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "y[%d] overlaps positions", i);
        a.weight[i] = weight ? weight[i] : nullptr;
        vec = vec && (((uintptr_t)x[i] | (uintptr_t)y[i] | (uintptr_t)a.weight[i]) & 15) == 0;
        a.rot.m[i] = RotaryMember{x[i], y[i], d_out / rotary->head_dim, d_out};
        a.rot.total_heads += d_out / rotary->head_dim;
    }
    DeviceGuard guard(ctx->device);
    hipStream_t s = (hipStream_t)stream;
    if ((rc = before_launch(ctx, s)))
        return rc;
    HIP_TRY(ctx, launch_norm_rotary(ctx->dtype == LORA_BF16, vec, a, s));
    return LORA_OK;
}

int do_cache_create(lora_ctx *ctx, lora_cache **out, int32_t kind, int32_t kv_heads, int32_t head_dim,
                    int32_t page_size, int32_t pages)
{
    if (out)
        *out = nullptr;
    if (check_ctx(ctx))
        return LORA_ERR_INVALID_ARGUMENT;
    ctx->last_error.clear();
    if (!out)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "out is NULL");
    if (kind != LORA_CACHE_NATIVE && kind != LORA_CACHE_FP8 && kind != LORA_CACHE_INT8)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "unknown kind %d", kind);
    if (kv_heads < 1 || kv_heads > kMostHeads)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "kv_heads %d not in 1..%d", kv_heads, kMostHeads);
    if (head_dim < 8 || head_dim > LORA_CACHE_MAX_DIM || head_dim % 8)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "head_dim %d is not a multiple of 8 in 8..%d", head_dim,
                    LORA_CACHE_MAX_DIM);
    if (page_size < kBlock || (page_size & (page_size - 1)))
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "page_size %d is not a power of two from %d on", page_size,
                    kBlock);
    if (pages < 1 || (int64_t)pages * page_size > INT32_MAX)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "%d pages of %d tokens are not 1..2^31 - 1 tokens", pages,
                    page_size);
    if (any_capture(ctx, nullptr))
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT,
                    "a cache is created while a stream this ctx launched on is under graph capture");
    std::unique_ptr<lora_cache> cache(new lora_cache);
    CacheView &v = cache->view;
    v.kind = kind;
    v.kv_heads = kv_heads;
    v.head_dim = head_dim;
    v.dp = padded_dim(head_dim);
    v.page_shift = 0;
    while (1 << v.page_shift < page_size)
        ++v.page_shift;
    v.pages = pages;
    v.elem = kind == LORA_CACHE_NATIVE ? ctx->elem : 1;
    v.half = kBlock * v.dp * v.elem;
    v.block = 2 * v.half + (kind == LORA_CACHE_NATIVE ? 0 : 2 * kBlock * (int)sizeof(float));
    const size_t bytes = (size_t)cache_block(v, pages, 0, 0);
    ctx->caches.reserve(ctx->caches.size() + 1);
    DeviceGuard guard(ctx->device);
    void *p = nullptr;
    int rc = device_alloc(ctx, &p, bytes, "cache");
    if (rc)
        return rc;
    v.base = (char *)p;
    hipError_t e = hipMemsetAsync(p, 0, bytes, ctx->side);
    if (e == hipSuccess)
        e = hipStreamSynchronize(ctx->side);
    if (e != hipSuccess) {
        ctx->allocations.pop_back();
        (void)hipFree(p);
        return hip_fail(ctx, e, "zeroing the cache");
    }
    *out = cache.get();
    ctx->caches.push_back(std::move(cache));
    return LORA_OK;
}

int do_cache_destroy(lora_ctx *ctx, lora_cache *cache)
{
    if (check_ctx(ctx))
        return LORA_ERR_INVALID_ARGUMENT;
    ctx->last_error.clear();
    if (!cache)
        return LORA_OK;
    int rc = check_cache(ctx, cache);
    if (rc)
        return rc;
    if (any_capture(ctx, nullptr))
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT,
                    "a cache is destroyed while a stream this ctx launched on is under graph capture");
    DeviceGuard guard(ctx->device);
    for (auto &st : ctx->streams)
        HIP_TRY(ctx, hipStreamSynchronize(st.stream));
    void *p = cache->view.base;
    ctx->allocations.erase(std::find(ctx->allocations.begin(), ctx->allocations.end(), p));
    ctx->caches.erase(std::find_if(ctx->caches.begin(), ctx->caches.end(),
                                   [&](const std::unique_ptr<lora_cache> &c) { return c.get() == cache; }));
    HIP_TRY(ctx, hipFree(p));
    return LORA_OK;
}

int do_cache_move(bool store, lora_ctx *ctx, const lora_cache *cache, const void *k, const void *v,
                  const int32_t *slots, int32_t n_tokens, void *stream)
{
    if (check_ctx(ctx))
        return LORA_ERR_INVALID_ARGUMENT;
    ctx->last_error.clear();
    int rc = check_cache(ctx, cache);
    if (rc || (rc = check_tokens(ctx, n_tokens)))
        return rc;
    if (n_tokens == 0)
        return LORA_OK;
    if (!k || !v || !slots)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "k, v or slots is NULL");
    CacheArgs a;
    std::memset(&a, 0, sizeof a);
    a.c = cache->view;
    a.slots = slots;
    a.T = n_tokens;
    a.flags = ctx->ws.plan.flags;
    if (store) {
        a.k_in = k;
        a.v_in = v;
    } else {
        const size_t bytes = (size_t)n_tokens * a.c.kv_heads * a.c.head_dim * ctx->elem;
        const size_t ids = sizeof(int32_t) * (size_t)n_tokens;
        if (overlap(k, bytes, v, bytes) || overlap(k, bytes, slots, ids) || overlap(v, bytes, slots, ids))
            return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "k, v and slots overlap");
        a.k_out = const_cast<void *>(k);
        a.v_out = const_cast<void *>(v);
    }
    DeviceGuard guard(ctx->device);
    hipStream_t s = (hipStream_t)stream;
    if ((rc = before_launch(ctx, s)))
        return rc;
    const bool bf16 = ctx->dtype == LORA_BF16;
    HIP_TRY(ctx, store ? launch_cache_store(bf16, a, s) : launch_cache_load(bf16, a, s));
    return LORA_OK;
}

// What one batch needs, cut from an allocation.
struct Cut {
    char *base;
    size_t used = 0;
    template <typename T>
    void take(T *&p, int64_t count)
    {
        p = base ? (T *)(base + used) : nullptr;
        used += ((size_t)count * sizeof(T) + 255) / 256 * 256;
    }
};

size_t cut_plan(char *base, AttendBatch &b)
{
    Cut c{base};
    c.take(b.plan, 1);
    for (int l = 0; l < 2; ++l) {
        c.take(b.tiles[l], b.cap[l]);
        c.take(b.start[l], kAttendWorkers);
    }
    c.take(b.list_before, (int64_t)b.n_seqs + 1);
    c.take(b.listed, b.n_tokens);
    c.take(b.prefix_tile, b.n_prefixes);
    return c.used;
}

size_t cut_parts(char *base, const AttendBatch &b, int dp, float *parts[2], float *sums[2])
{
    Cut c{base};
    for (int l = 0; l < 2; ++l) {
        const int64_t rows = b.cap[l] ? part_slots(b.workers[l], b.kept_cap[l], b.kv_heads) * list_rows(l) : 0;
        c.take(sums[l], rows * 2);
        c.take(parts[l], rows * dp);
    }
    return c.used;
}

// Not at every batch that is a little larger; all that came before stay below this one.
size_t grown(size_t need, size_t have) { return (std::max(need + need / 4, 2 * have) + 255) / 256 * 256; }

int do_attend_prepare(lora_ctx *ctx, const lora_cache *cache, int32_t q_heads, const lora_attend_batch *batch,
                      void *stream)
{
    if (check_ctx(ctx))
        return LORA_ERR_INVALID_ARGUMENT;
    ctx->last_error.clear();
    int rc = check_cache(ctx, cache);
    if (rc)
        return rc;
    if (!batch)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "batch is NULL");
    if ((rc = check_tokens(ctx, batch->n_tokens)))
        return rc;
    const CacheView &v = cache->view;
    if (q_heads < 1 || q_heads > kMostHeads || q_heads % v.kv_heads)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "q_heads %d is not a multiple of kv_heads %d, up to %d", q_heads,
                    v.kv_heads, kMostHeads);
    if ((int64_t)batch->n_tokens * q_heads > INT32_MAX)
        return fail(ctx, LORA_ERR_TOO_MANY_TOKENS, "%d tokens of %d heads are more than 2^31 - 1 rows",
                    batch->n_tokens, q_heads);
    if (batch->n_seqs < 0 || batch->n_prefixes < 0 || batch->max_pages < 0 || batch->prefix_max_pages < 0)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "a size of the batch is negative");
    if (batch->n_seqs > LORA_ATTEND_MAX_SEQS || batch->n_prefixes > LORA_ATTEND_MAX_PREFIXES)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT,
                    "%d requests or %d prefixes exceed LORA_ATTEND_MAX_SEQS or LORA_ATTEND_MAX_PREFIXES",
                    batch->n_seqs, batch->n_prefixes);
    if (batch->max_queries < 1)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "max_queries %d < 1", batch->max_queries);
    if (batch->n_seqs && (!batch->lengths || (batch->max_pages && !batch->pages)))
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "lengths or pages is NULL");
    if (!batch->q_start && batch->n_seqs > batch->n_tokens)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "%d requests without q_start, but %d tokens", batch->n_seqs,
                    batch->n_tokens);
    if (batch->n_prefixes && (!batch->prefix_seqs || !batch->prefix_lengths ||
                              (batch->prefix_max_pages && !batch->prefix_pages)))
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "prefix_seqs, prefix_lengths or prefix_pages is NULL");

    AttendState &st = ctx->attend;
    AttendBatch b;
    std::memset(&b, 0, sizeof b);
    b.q_start = batch->q_start;
    b.lengths = batch->lengths;
    b.pages = batch->pages;
    b.prefix_seqs = batch->prefix_seqs;
    b.prefix_lengths = batch->prefix_lengths;
    b.prefix_pages = batch->prefix_pages;
    b.n_tokens = batch->n_tokens;
    b.n_seqs = batch->n_seqs;
    b.n_prefixes = batch->n_prefixes;
    b.max_pages = batch->max_pages;
    b.prefix_max_pages = batch->prefix_max_pages;
    b.max_queries = std::min(batch->max_queries, std::max(batch->n_tokens, 1));
    set_group(b, q_heads / v.kv_heads);
    b.kv_heads = v.kv_heads;
    b.page_shift = v.page_shift;
    b.wide = ctx->dtype == LORA_BF16;
    b.workers[0] = kAttendCus * kAttendPerCu(ctx->elem, v.kind, v.dp);
    b.workers[1] = kAttendCus * (v.dp <= 128 ? 2 : 1);
    b.flags = ctx->ws.plan.flags;
    if (b.n_tokens && b.n_seqs) {
        if (!size_batch(b))
            return fail(ctx, LORA_ERR_TOO_MANY_TOKENS, "the batch needs more than 2^27 tiles");
        float *parts[2], *sums[2];
        const size_t plan = cut_plan(nullptr, b), rest = cut_parts(nullptr, b, v.dp, parts, sums);
        DeviceGuard guard(ctx->device);
        hipStream_t s = (hipStream_t)stream;
        if ((plan > st.plan_bytes || rest > st.parts_bytes) && any_capture(ctx, s))
            return fail(ctx, LORA_ERR_INVALID_ARGUMENT,
                        "the workspace must grow to %zu bytes: prepare a batch of these sizes once before "
                        "the capture", 2 * plan + rest);
        void *p = nullptr;
        if (plan > st.plan_bytes) {
            const size_t more = grown(plan, st.plan_bytes);
            if ((rc = device_alloc(ctx, &p, 2 * more, "attention plans")))
                return rc;
            st.plans = (char *)p;
            st.plan_bytes = more;
        }
        if (rest > st.parts_bytes) {
            const size_t more = grown(rest, st.parts_bytes);
            if ((rc = device_alloc(ctx, &p, more, "attention parts")))
                return rc;
            st.parts_base = (char *)p;
            st.parts_bytes = more;
        }
        cut_plan(st.plans + (capture_of(s) ? st.plan_bytes : 0), b);
        cut_parts(st.parts_base, b, v.dp, parts, sums);
        if ((rc = before_launch(ctx, s)))
            return rc;
        st.prepared = false;
        if (!b.simple)
            HIP_TRY(ctx, launch_attend_plan(b, s));
        for (int l = 0; l < 2; ++l) {
            st.parts[l] = parts[l];
            st.sums[l] = sums[l];
        }
    }
    st.capture = capture_of((hipStream_t)stream);
    st.batch = b;
    st.head_dim = v.head_dim;
    st.prepared = true;
    return LORA_OK;
}

int do_attend(lora_ctx *ctx, const lora_cache *cache, const void *q, void *y, double scale, void *stream)
{
    if (check_ctx(ctx))
        return LORA_ERR_INVALID_ARGUMENT;
    ctx->last_error.clear();
    int rc = check_cache(ctx, cache);
    if (rc)
        return rc;
    const AttendState &st = ctx->attend;
    if (!st.prepared)
        return fail(ctx, LORA_ERR_NO_PLAN, "no batch prepared (lora_attend_prepare)");
    const CacheView &v = cache->view;
    const AttendBatch &b = st.batch;
    if (v.kv_heads != b.kv_heads || v.head_dim != st.head_dim || v.page_shift != b.page_shift)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "the batch was prepared for a cache of another shape");
    const float s2 = (float)(scale * 1.4426950408889634073599246810019);
    if (!(scale > 0.0) || !std::isfinite(s2) || s2 == 0.f)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "scale must be positive and finite");
    if (!b.n_tokens || !b.n_seqs)
        return LORA_OK;
    // the plan that a captured launch finds at a replay must be its own
    if (capture_of((hipStream_t)stream) != st.capture)
        return fail(ctx, LORA_ERR_NO_PLAN, "the batch was prepared %s",
                    st.capture ? "in a capture that this call is not part of"
                               : "outside of the capture that this call is part of");
    if (!q || !y)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "q or y is NULL");
    const size_t bytes = (size_t)b.n_tokens * b.group * b.kv_heads * v.head_dim * ctx->elem;
    if (overlap(q, bytes, y, bytes))
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "y overlaps q");
    AttendArgs a;
    std::memset(&a, 0, sizeof a);
    a.b = b;
    a.c = v;
    a.q = q;
    a.y = y;
    a.scale = s2;
    for (int l = 0; l < 2; ++l) {
        a.parts[l] = st.parts[l];
        a.sums[l] = st.sums[l];
    }
    DeviceGuard guard(ctx->device);
    hipStream_t s = (hipStream_t)stream;
    if ((rc = before_launch(ctx, s)))
        return rc;
    HIP_TRY(ctx, launch_attend(ctx->dtype == LORA_BF16, a, s));
    return LORA_OK;
}

}  // namespace

extern "C" {

int lora_norm_rotary_group(lora_ctx *ctx, const lora_rotary *rotary, int32_t n, const int32_t *modules,
                           const void *const *x, const void *const *weight, double eps, void *const *y,
                           const int32_t *positions, int32_t n_tokens, void *stream)
{
    return guarded([&] { return do_norm_rotary(ctx, rotary, n, modules, x, weight, eps, y, positions, n_tokens, stream); });
}

int lora_cache_create(lora_ctx *ctx, lora_cache **out, int32_t kind, int32_t kv_heads, int32_t head_dim,
                      int32_t page_size, int32_t pages)
{
    return guarded([&] { return do_cache_create(ctx, out, kind, kv_heads, head_dim, page_size, pages); });
}

int lora_cache_destroy(lora_ctx *ctx, lora_cache *cache)
{
    return guarded([&] { return do_cache_destroy(ctx, cache); });
}

int lora_cache_store(lora_ctx *ctx, lora_cache *cache, const void *k, const void *v, const int32_t *slots,
                     int32_t n_tokens, void *stream)
{
    return guarded([&] { return do_cache_move(true, ctx, cache, k, v, slots, n_tokens, stream); });
}

int lora_cache_load(lora_ctx *ctx, const lora_cache *cache, const int32_t *slots, void *k, void *v,
                    int32_t n_tokens, void *stream)
{
    return guarded([&] { return do_cache_move(false, ctx, cache, k, v, slots, n_tokens, stream); });
}

int lora_attend_prepare(lora_ctx *ctx, const lora_cache *cache, int32_t q_heads, const lora_attend_batch *batch,
                        void *stream)
{
    return guarded([&] { return do_attend_prepare(ctx, cache, q_heads, batch, stream); });
}

int lora_attend(lora_ctx *ctx, const lora_cache *cache, const void *q, void *y, double scale, void *stream)
{
    return guarded([&] { return do_attend(ctx, cache, q, y, scale, stream); });
}

}  // extern "C"
