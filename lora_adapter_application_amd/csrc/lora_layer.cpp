// lora_layer.cpp -- the C ABI of a layer's frozen part, declared in
// include/lora_mi355x.h: 4-bit base weights and their products
// (lora_base_*), and rotary positions (lora_rotary_*).
//
// Base weights belong to the ctx's modules.  They have the ctx's ordering
// without host synchronisation, apart from that of the slots: a load runs on the
// side stream and records an event of its own, which the stream of every later
// base product waits for once; before it overwrites weights the side stream waits
// for the tail of each stream that has launched a base product since the last base
// load.  A slot load waits for a stream only if that has read slots since the last one (and
// then for all that is on it), and base products wait for no slot load: the adapters that a
// step misses can be uploaded under its base products.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/lora_mi355x.h"
#include "lora_ctx.h"
#include "lora_layer.h"

using namespace lora;

namespace {

int64_t pad(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Rows of `bytes` starting at p and q share memory.
bool overlap(const void *p, size_t pb, const void *q, size_t qb)
{
    return (uintptr_t)p < (uintptr_t)q + qb && (uintptr_t)q < (uintptr_t)p + pb;
}

// Make stream s wait for the base loads issued so far.  Under capture the load
// event, recorded outside the capture, cannot be waited for: loads must be complete.
int before_layer_launch(lora_ctx *c, hipStream_t s, bool reads_base)
{
    StreamState *st = stream_state(c, s);
    if (!st)
        return fail(c, LORA_ERR_HIP, "hipEventCreateWithFlags failed");
    if (reads_base && st->base_waited < c->base_gen && c->base_synced < c->base_gen) {
        if (stream_capturing(s))
            return fail(c, LORA_ERR_INVALID_ARGUMENT,
                        "base loads pending on a stream under graph capture: call lora_sync_loads "
                        "before the capture");
        HIP_TRY(c, hipStreamWaitEvent(s, c->base_done, 0));
        st->base_waited = c->base_gen;
    }
    if (reads_base)
        st->base_since_load = true;
    st->since_fence = true;
    return LORA_OK;
}

int check_tokens(lora_ctx *c, int32_t n_tokens)
{
    if (n_tokens < 0)
        return fail(c, LORA_ERR_INVALID_ARGUMENT, "n_tokens %d < 0", n_tokens);
    if (n_tokens > c->max_tokens)
        return fail(c, LORA_ERR_TOO_MANY_TOKENS, "n_tokens %d > max_tokens %d", n_tokens,
                    c->max_tokens);
    return LORA_OK;
}

int check_base(lora_ctx *c, int32_t module)
{
    if (module < 0 || module >= c->n_modules)
        return fail(c, LORA_ERR_BAD_MODULE, "module %d not in 0..%d", module, c->n_modules - 1);
    if ((size_t)module >= c->base.size() || !c->base[module].spb)
        return fail(c, LORA_ERR_INVALID_ARGUMENT, "module %d has no base weight (lora_base_load)",
                    module);
    return LORA_OK;
}

BaseMember base_member(const lora_ctx *c, int32_t module, const void *x, const void *add, void *y)
{
    const BasePack &p = c->base[module];
    const lora_module_shape sh = c->shapes[module];
    BaseMember m{};
    m.q = p.q;
    m.sc = p.sc();
    m.bias = p.has_bias ? p.bias : nullptr;
    m.x = x;
    m.add = add;
    m.y = y;
    m.d_in = sh.d_in;
    m.d_out = sh.d_out;
    m.kb = ceil_div(sh.d_in, kBaseK);
    m.has_zero = p.has_zero;
    return m;
}

// What a launch on s may take for granted of the zero points of n modules: a captured one
// only what no later load can change.
Zeros zeros_of(const lora_ctx *c, int32_t n, const int32_t *modules, int spb, hipStream_t s)
{
    for (int i = 0; i < n; ++i)
        if (c->base[modules[i]].spb == spb && c->base[modules[i]].zero)
            return kZerosSome;
    return s && stream_capturing(s) ? kZerosAsk : kZerosNone;
}

// Device memory the ctx keeps until it is destroyed.
int base_alloc(lora_ctx *c, void **p, size_t bytes, int32_t module)
{
    c->allocations.reserve(c->allocations.size() + 1);
    const hipError_t e = hipMalloc(p, bytes);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        *p = nullptr;
        return fail(c, (e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation)
                           ? LORA_ERR_OUT_OF_MEMORY : LORA_ERR_HIP,
                    "base weight of module %d (%zu bytes): %s", module, bytes, hipGetErrorString(e));
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

int do_base_load(lora_ctx *ctx, int32_t module, const void *q, const float *scale,
                   const uint8_t *zero, int32_t group_size, const void *bias)
{
    if (check_ctx(ctx))
        return LORA_ERR_INVALID_ARGUMENT;
    ctx->last_error.clear();
    if (module < 0 || module >= ctx->n_modules)
        return fail(ctx, LORA_ERR_BAD_MODULE, "module %d not in 0..%d", module, ctx->n_modules - 1);
    if (!q || !scale)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "q or scale is NULL");
    if (group_size < 0 || (group_size != 32 && group_size != 64 && group_size % 128))
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT,
                    "group_size %d is not 0, 32, 64 or a multiple of 128", group_size);
    DeviceGuard guard(ctx->device);
    const void *src[4] = {q, scale, zero, bias};
    bool local[4] = {false, false, false, false};     // read by the pack kernel where it is
    for (int i = 0; i < 4; ++i) {
        if (!src[i])
            continue;
        if (check_source(src[i], ctx->device))
            return fail(ctx, LORA_ERR_HOST_NOT_PINNED,
                        "base weight of module %d must be in pinned host or device memory", module);
        hipPointerAttribute_t attr;
        if (hipPointerGetAttributes(&attr, src[i]) == hipSuccess)
            local[i] = attr.type == hipMemoryTypeDevice && attr.device == ctx->device &&
                       ((uintptr_t)src[i] & 3) == 0;
    }
    for (auto &st : ctx->streams)
        if (stream_capturing(st.stream))
            return fail(ctx, LORA_ERR_INVALID_ARGUMENT,
                        "base load while a stream this ctx launched on is under graph capture");
    const lora_module_shape sh = ctx->shapes[module];
    if (sh.d_in > kBaseMaxIn)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "d_in %d of module %d exceeds %d", sh.d_in, module,
                    kBaseMaxIn);
    const bool bf16 = ctx->dtype == LORA_BF16;
    const int64_t kb = ceil_div(sh.d_in, kBaseK), nb = ceil_div(sh.d_out, kBaseCols);
    const int group = group_size ? group_size : (int)pad(sh.d_in, kBaseK);
    const int groups = ceil_div(sh.d_in, group);
    const int spb = group >= kBaseK ? 1 : kBaseK / group;
    const size_t word = bf16 ? 4 : 8;
    if (!ctx->base_done)
        HIP_TRY(ctx, hipEventCreateWithFlags(&ctx->base_done, hipEventDisableTiming));
    if (ctx->base.empty())
        ctx->base.resize(ctx->n_modules);
    BasePack &p = ctx->base[module];
    // Storage first, each kind kept for the module's next load: a failed allocation leaves the
    // weight as it was.
    void *nq = p.q, *nsc = p.sc(spb), *nbias = p.bias;
    int rc;
    if (!nq && (rc = base_alloc(ctx, &nq, (size_t)(nb * kb) * 1024 + 16, module)))
        return rc;
    p.q = (uint32_t *)nq;
    p.has_zero = p.q + nb * kb * 256;
    if (!nsc) {
        if ((rc = base_alloc(ctx, &nsc, (size_t)(nb * kb) * kBaseCols * spb * word, module)))
            return rc;
        p.sc(spb) = nsc;
    }
    if (bias && !nbias) {
        if ((rc = base_alloc(ctx, &nbias, (size_t)sh.d_out * ctx->elem, module)))
            return rc;
        p.bias = nbias;
    }
    for (auto &st : ctx->streams) {
        if (!st.base_since_load)
            continue;
        HIP_TRY(ctx, hipEventRecord(st.tail, st.stream));
        HIP_TRY(ctx, hipStreamWaitEvent(ctx->side, st.tail, 0));
        st.base_since_load = false;
    }
    // Weights on this device are repacked from where they are, others through the
    // ctx's stage, as many rows at a time as it takes (16 at least: it holds 16 (d_in + d_out)
    // elements of 2 or 4 bytes, 32 d_in + 256 or more, and 16 rows with groups of 32 or more
    // need at most 16 (d_in / 2 + 5 (d_in / 32 + 1)) + 48, under 11 d_in + 128).
    const int64_t row_q = sh.d_in / 2, row_s = 4ll * groups, row_z = zero ? groups : 0;
    int64_t row_bytes = (local[0] ? 0 : row_q) + (local[1] ? 0 : row_s) + (local[2] ? 0 : row_z);
    int64_t rows = sh.d_out;
    if (row_bytes) {
        const int64_t room = ctx->stage_elems * ctx->elem - 3 * 16;
        rows = std::min<int64_t>(rows, room / row_bytes / kBaseCols * kBaseCols);
        if (rows < std::min<int64_t>(kBaseCols, sh.d_out))
            return fail(ctx, LORA_ERR_OUT_OF_MEMORY, "the stage holds no 16 rows of module %d", module);
    }
    // from the first copy to the event the module has no weight: a load that fails between
    // leaves none, not part of one and part of another
    p.spb = 0;
    for (int64_t r0 = 0; r0 < sh.d_out; r0 += rows) {
        const int64_t n = std::min<int64_t>(rows, sh.d_out - r0);
        char *stage = (char *)ctx->stage;
        const void *at[3];
        const int64_t per[3] = {row_q, row_s, row_z};
        for (int i = 0; i < 3; ++i) {
            at[i] = src[i] ? (const char *)src[i] + r0 * per[i] : nullptr;
            if (!src[i] || local[i])
                continue;
            HIP_TRY(ctx, hipMemcpyAsync(stage, at[i], (size_t)(n * per[i]), hipMemcpyDefault, ctx->side));
            at[i] = stage;
            stage += pad(n * per[i], 16);
        }
        BasePackArgs a{};
        a.q = (const uint8_t *)at[0];
        a.scale = (const float *)at[1];
        a.zero = (const uint8_t *)at[2];
        a.q_out = p.q + (r0 / kBaseCols) * kb * 256;
        a.has_zero = p.has_zero;
        a.sc_out = (char *)nsc + (size_t)(r0 / kBaseCols) * kb * kBaseCols * spb * word;
        a.rows = (int32_t)n;
        a.d_in = sh.d_in;
        a.group = group;
        a.groups = groups;
        a.spb = spb;
        HIP_TRY(ctx, launch_base_pack(bf16, a, ctx->side));
    }
    if (bias)
        HIP_TRY(ctx, hipMemcpyAsync(p.bias, bias, (size_t)sh.d_out * ctx->elem, hipMemcpyDefault,
                                    ctx->side));
    HIP_TRY(ctx, hipEventRecord(ctx->base_done, ctx->side));
    ctx->base_gen += 1;
    p.spb = spb;
    p.has_bias = bias != nullptr;
    p.zero = zero != nullptr;
    return LORA_OK;
}

int do_base_group(lora_ctx *ctx, int32_t n, const int32_t *modules, const void *const *x,
                    const void *const *add, void *const *y, int32_t n_tokens, void *stream)
{
    if (check_ctx(ctx))
        return LORA_ERR_INVALID_ARGUMENT;
    ctx->last_error.clear();
    int rc = check_group(ctx, n, modules);
    for (int i = 0; !rc && i < n; ++i)
        rc = check_base(ctx, modules[i]);
    if (rc || (rc = check_tokens(ctx, n_tokens)))
        return rc;
    if (n_tokens == 0)
        return LORA_OK;
    if ((rc = check_ptrs(ctx, n, x, "x", false)) ||
        (rc = check_ptrs(ctx, n, (const void *const *)y, "y", true)))
        return rc;
    size_t xb[kMaxGroup], yb[kMaxGroup];
    for (int i = 0; i < n; ++i) {
        xb[i] = (size_t)n_tokens * ctx->shapes[modules[i]].d_in * ctx->elem;
        yb[i] = (size_t)n_tokens * ctx->shapes[modules[i]].d_out * ctx->elem;
    }
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            const void *aj = add ? add[j] : nullptr;
            if (overlap(y[i], yb[i], x[j], xb[j]) || (j != i && overlap(y[i], yb[i], y[j], yb[j])) ||
                (aj && !(j == i && aj == y[i]) && overlap(y[i], yb[i], aj, yb[j])))
                return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "y[%d] overlaps x, add or y of member %d",
                            i, j);
        }
    DeviceGuard guard(ctx->device);
    hipStream_t s = (hipStream_t)stream;
    if ((rc = before_layer_launch(ctx, s, true)))
        return rc;
    for (int spb = 1; spb <= 4; spb *= 2) {
        BaseArgs a;
        std::memset(&a, 0, sizeof a);
        a.T = n_tokens;
        for (int i = 0; i < n; ++i) {
            if (ctx->base[modules[i]].spb != spb)
                continue;
            a.m[a.n++] = base_member(ctx, modules[i], x[i], add ? add[i] : nullptr, y[i]);
        }
        if (!a.n)
            continue;
        a.zeros = zeros_of(ctx, n, modules, spb, s);
        HIP_TRY(ctx, launch_base(ctx->dtype == LORA_BF16, false, spb, a, s));
    }
    return LORA_OK;
}

int do_base(lora_ctx *ctx, const void *x, const void *add, void *y, int32_t n_tokens,
              int32_t module, void *stream)
{
    return do_base_group(ctx, 1, &module, &x, &add, &y, n_tokens, stream);
}

int do_base_gated(lora_ctx *ctx, int32_t gate_module, int32_t up_module, const void *x,
                    const void *gate_add, const void *up_add, void *y, int32_t n_tokens,
                    int32_t activation, void *stream)
{
    if (check_ctx(ctx))
        return LORA_ERR_INVALID_ARGUMENT;
    ctx->last_error.clear();
    int rc = check_base(ctx, gate_module);
    if (rc || (rc = check_base(ctx, up_module)) || (rc = check_tokens(ctx, n_tokens)))
        return rc;
    const lora_module_shape sg = ctx->shapes[gate_module], su = ctx->shapes[up_module];
    if (sg.d_in != su.d_in || sg.d_out != su.d_out)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "modules %d and %d have different shapes",
                    gate_module, up_module);
    if (ctx->base[gate_module].spb != ctx->base[up_module].spb)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT,
                    "the base weights of modules %d and %d have different group storage",
                    gate_module, up_module);
    if (activation < LORA_ACT_SILU || activation > LORA_ACT_GELU_TANH)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "unknown activation %d", activation);
    if (n_tokens == 0)
        return LORA_OK;
    if (!x || !y)
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "x or y is NULL");
    const size_t xb = (size_t)n_tokens * sg.d_in * ctx->elem, yb = (size_t)n_tokens * sg.d_out * ctx->elem;
    const void *adds[2] = {gate_add, up_add};
    if (overlap(y, yb, x, xb))
        return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "y overlaps x");
    for (const void *a : adds)
        if (a && a != y && overlap(y, yb, a, yb))
            return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "y overlaps an add buffer that it is not");
    DeviceGuard guard(ctx->device);
    hipStream_t s = (hipStream_t)stream;
    if ((rc = before_layer_launch(ctx, s, true)))
        return rc;
    BaseArgs a;
    std::memset(&a, 0, sizeof a);
    a.n = 2;
    a.T = n_tokens;
    a.act = activation;
    a.m[0] = base_member(ctx, gate_module, x, gate_add, y);
    a.m[1] = base_member(ctx, up_module, x, up_add, y);
    const int32_t both[2] = {gate_module, up_module};
    a.zeros = zeros_of(ctx, 2, both, ctx->base[gate_module].spb, s);
    HIP_TRY(ctx, launch_base(ctx->dtype == LORA_BF16, true, ctx->base[gate_module].spb, a, s));
    return LORA_OK;
}

int do_rotary_init(lora_rotary *out, const lora_rotary_params *p)
{
    fail(nullptr, 0, "%s", "");
    auto bad = [](const char *what) { return fail(nullptr, LORA_ERR_INVALID_ARGUMENT, "%s", what); };
    if (!out || !p)
        return bad("out or params is NULL");
    if (p->head_dim < 2 || p->head_dim % 2)
        return bad("head_dim must be even and positive");
    if (p->rotary_dim < 2 || p->rotary_dim % 2 || p->rotary_dim > p->head_dim ||
        p->rotary_dim > LORA_ROTARY_MAX_DIM)
        return bad("rotary_dim must be even, in 2..min(head_dim, LORA_ROTARY_MAX_DIM)");
    if (p->layout != LORA_ROTARY_HALF && p->layout != LORA_ROTARY_INTERLEAVED)
        return bad("unknown layout");
    if (p->scaling < LORA_ROTARY_SCALE_NONE || p->scaling > LORA_ROTARY_SCALE_BANDED)
        return bad("unknown scaling");
    if (!(p->base > 1.0) || !std::isfinite(p->base))
        return bad("base must be finite and above 1");
    const bool yarn = p->scaling == LORA_ROTARY_SCALE_YARN;
    const bool banded = p->scaling == LORA_ROTARY_SCALE_BANDED;
    if (p->scaling != LORA_ROTARY_SCALE_NONE && (!(p->factor >= 1.0) || !std::isfinite(p->factor)))
        return bad("factor must be finite and at least 1");
    if ((yarn || banded) && (!(p->original_positions > 0.0) || !std::isfinite(p->original_positions)))
        return bad("original_positions must be finite and positive");
    if (yarn && (!(p->beta_slow > 0.0) || !(p->beta_fast > p->beta_slow) || !std::isfinite(p->beta_fast)))
        return bad("beta_fast > beta_slow > 0 is needed");
    if (yarn && (!(p->attention_factor >= 0.0) || !std::isfinite(p->attention_factor)))
        return bad("attention_factor must be finite and not negative");
    if (banded && (!(p->low_factor > 0.0) || !(p->high_factor > p->low_factor) ||
                   !std::isfinite(p->high_factor)))
        return bad("high_factor > low_factor > 0 is needed");
    const double tau = 6.283185307179586476925286766559;
    const int dim = p->rotary_dim;
    std::memset(out, 0, sizeof *out);
    out->head_dim = p->head_dim;
    out->rotary_dim = dim;
    out->layout = p->layout;
    out->amplitude = 1.f;
    double low = 0, high = 0;
    if (yarn) {
        // the pair index at which original_positions hold `turns` turns
        auto index = [&](double turns) {
            return dim * std::log(p->original_positions / (turns * tau)) / (2.0 * std::log(p->base));
        };
        low = std::max(std::floor(index(p->beta_fast)), 0.0);
        high = std::min(std::ceil(index(p->beta_slow)), dim - 1.0);
        const double f = p->attention_factor > 0.0 ? p->attention_factor : 0.1 * std::log(p->factor) + 1.0;
        out->amplitude = (float)f;
        if (!std::isfinite(out->amplitude))
            return bad("attention_factor does not fit fp32");
    }
    for (int i = 0; i < dim / 2; ++i) {
        const double rate = std::pow(p->base, -2.0 * i / dim);
        double keep = 1.0;                            // share of the unscaled rate
        if (p->scaling == LORA_ROTARY_SCALE_LINEAR)
            keep = 0.0;
        else if (yarn)                                // a ramp of no width is a step
            keep = 1.0 - std::min(std::max((i - low) / std::max(high - low, 1e-3), 0.0), 1.0);
        else if (banded)
            keep = std::min(std::max((p->original_positions * rate / tau - p->low_factor) /
                                         (p->high_factor - p->low_factor), 0.0), 1.0);
        const double slow = p->scaling == LORA_ROTARY_SCALE_NONE ? rate : rate / p->factor;
        out->turns[i] = (slow * (1.0 - keep) + rate * keep) / tau;
    }
    return LORA_OK;
}

int do_rotary_group(lora_ctx *ctx, const lora_rotary *rotary, int32_t n, const int32_t *modules,
                      const void *const *x, void *const *y, const int32_t *positions,
                      int32_t n_tokens, void *stream)
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
    RotaryArgs a;
    std::memset(&a, 0, sizeof a);
    a.rot = *rotary;
    a.n = n;
    a.T = n_tokens;
    a.positions = positions;
    const int V = 16 / ctx->elem;
    const int pairs = rotary->rotary_dim / 2;
    bool vec = rotary->head_dim % V == 0 && rotary->rotary_dim % V == 0 &&
               (rotary->layout == LORA_ROTARY_INTERLEAVED || pairs % V == 0);
    for (int i = 0; i < n; ++i) {
        const int d_out = ctx->shapes[modules[i]].d_out;
        const size_t bytes = (size_t)n_tokens * d_out * ctx->elem;
        for (int j = 0; j < n; ++j) {
            const size_t other = (size_t)n_tokens * ctx->shapes[modules[j]].d_out * ctx->elem;
            if ((!(i == j && x[j] == y[i]) && overlap(y[i], bytes, x[j], other)) ||
                (i != j && overlap(y[i], bytes, y[j], other)))
                return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "y[%d] overlaps x or y of member %d", i, j);
        }
        if (overlap(y[i], bytes, positions, sizeof(int32_t) * (size_t)n_tokens))
            return fail(ctx, LORA_ERR_INVALID_ARGUMENT, "y[%d] overlaps positions", i);
        vec = vec && (((uintptr_t)x[i] | (uintptr_t)y[i]) & 15) == 0;
        a.m[i] = RotaryMember{x[i], y[i], d_out / rotary->head_dim, d_out};
        a.total_heads += d_out / rotary->head_dim;
    }
    DeviceGuard guard(ctx->device);
    hipStream_t s = (hipStream_t)stream;
    if ((rc = before_layer_launch(ctx, s, false)))
        return rc;
    HIP_TRY(ctx, launch_rotary(ctx->dtype == LORA_BF16, vec, a, s));
    return LORA_OK;
}

}  // namespace

extern "C" {

int lora_base_load(lora_ctx *ctx, int32_t module, const void *q, const float *scale,
                   const uint8_t *zero, int32_t group_size, const void *bias)
{
    return guarded([&] { return do_base_load(ctx, module, q, scale, zero, group_size, bias); });
}

int lora_base_group(lora_ctx *ctx, int32_t n, const int32_t *modules, const void *const *x,
                    const void *const *add, void *const *y, int32_t n_tokens, void *stream)
{
    return guarded([&] { return do_base_group(ctx, n, modules, x, add, y, n_tokens, stream); });
}

int lora_base(lora_ctx *ctx, const void *x, const void *add, void *y, int32_t n_tokens,
              int32_t module, void *stream)
{
    return guarded([&] { return do_base(ctx, x, add, y, n_tokens, module, stream); });
}

int lora_base_gated(lora_ctx *ctx, int32_t gate_module, int32_t up_module, const void *x,
                    const void *gate_add, const void *up_add, void *y, int32_t n_tokens,
                    int32_t activation, void *stream)
{
    return guarded([&] { return do_base_gated(ctx, gate_module, up_module, x, gate_add, up_add, y, n_tokens, activation, stream); });
}

int lora_rotary_init(lora_rotary *out, const lora_rotary_params *p)
{
    return guarded([&] { return do_rotary_init(out, p); });
}

int lora_rotary_group(lora_ctx *ctx, const lora_rotary *rotary, int32_t n, const int32_t *modules,
                      const void *const *x, void *const *y, const int32_t *positions,
                      int32_t n_tokens, void *stream)
{
    return guarded([&] { return do_rotary_group(ctx, rotary, n, modules, x, y, positions, n_tokens, stream); });
}

}  // extern "C"
