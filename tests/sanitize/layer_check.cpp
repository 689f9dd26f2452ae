// layer_check.cpp -- drives the host side of a layer's frozen part
// (lora_adapter_application_amd/csrc/lora_layer.cpp) under AddressSanitizer and
// UndefinedBehaviorSanitizer without a GPU: rotary rates over many settings, and
// every refusal that needs no device.  The kernels' launch functions are stubs
// that must not be reached.  Built and run by tests/test_layer_sanitizers.py.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>

#include "lora_mi355x.h"
#include "../../lora_adapter_application_amd/csrc/lora_layer.h"

static int failures = 0;

namespace lora {
static hipError_t reached()
{
    std::printf("FAIL a launch was reached\n");
    ++failures;
    return hipErrorNotSupported;
}
hipError_t launch_plan(const int32_t *, int32_t, int32_t, const PlanBuffers &, hipStream_t,
                       const LaunchTiming *) { return reached(); }
hipError_t launch_shrink(bool, const ShrinkArgs &, const SlotMeta &, hipStream_t, const LaunchTiming &)
{ return reached(); }
hipError_t launch_expand(bool, const ExpandArgs &, const SlotMeta &, hipStream_t, const LaunchTiming &)
{ return reached(); }
hipError_t launch_fused(const FusedArgs &, const SlotMeta &, hipStream_t, const LaunchTiming &)
{ return reached(); }
hipError_t launch_slot_finalize(bool, const FinalizeBatch &, hipStream_t) { return reached(); }
hipError_t launch_saved(bool, const SavedArgs &, hipStream_t, const LaunchTiming &) { return reached(); }
hipError_t scratch_address(int, void **) { return reached(); }
hipError_t xcd_dispatch_check(int, hipStream_t, bool *) { return reached(); }
hipError_t launch_base_pack(bool, const BasePackArgs &, hipStream_t) { return reached(); }
hipError_t launch_base(bool, bool, int, const BaseArgs &, hipStream_t) { return reached(); }
hipError_t launch_rotary(bool, bool, const RotaryArgs &, hipStream_t) { return reached(); }
}  // namespace lora

static void expect(int got, int want, const char *what)
{
    if (got != want) {
        std::printf("FAIL %s: status %d, expected %d (%s)\n", what, got, want, lora_last_error(nullptr));
        ++failures;
    }
}

int main()
{
    const int bad = LORA_ERR_INVALID_ARGUMENT;
    lora_rotary rot;
    lora_rotary_params p;
    std::memset(&p, 0, sizeof p);
    p.head_dim = p.rotary_dim = 128;
    p.base = 10000.0;
    p.factor = 8.0;
    p.original_positions = 8192;
    p.beta_fast = 32;
    p.beta_slow = 1;
    p.low_factor = 1;
    p.high_factor = 4;
    for (int dim = 2; dim <= LORA_ROTARY_MAX_DIM; dim += 2)
        for (int scaling = 0; scaling < 4; ++scaling)
            for (double base : {1.5, 10000.0, 1e12})
                for (double orig : {1e-6, 512.0, 1e15}) {
                    p.head_dim = p.rotary_dim = dim;
                    p.scaling = scaling;
                    p.base = base;
                    p.original_positions = orig;
                    expect(lora_rotary_init(&rot, &p), LORA_OK, "rotary_init");
                    for (int i = 0; i < LORA_ROTARY_MAX_DIM / 2; ++i)
                        if (!std::isfinite(rot.turns[i]) || rot.turns[i] < 0 || (i >= dim / 2 && rot.turns[i] != 0)) {
                            std::printf("FAIL turns[%d] = %g (dim %d scaling %d)\n", i, rot.turns[i], dim, scaling);
                            ++failures;
                        }
                }
    const double nan = std::nan(""), inf = std::numeric_limits<double>::infinity();
    auto with = [&](auto change, const char *what) {
        lora_rotary_params q = p;
        q.head_dim = q.rotary_dim = 64;
        q.scaling = LORA_ROTARY_SCALE_YARN;
        q.base = 10000;
        q.original_positions = 4096;
        change(q);
        expect(lora_rotary_init(&rot, &q), bad, what);
    };
    with([&](auto &q) { q.head_dim = INT32_MIN; }, "head_dim");
    with([&](auto &q) { q.rotary_dim = INT32_MAX - 1; }, "rotary_dim");
    with([&](auto &q) { q.layout = INT32_MAX; }, "layout");
    with([&](auto &q) { q.scaling = INT32_MIN; }, "scaling");
    for (double v : {nan, inf, -inf, 0.0, 1.0})
        with([&](auto &q) { q.base = v; }, "base");
    for (double v : {nan, inf, -inf, 0.0})
        with([&](auto &q) { q.factor = v; }, "factor");
    for (double v : {nan, inf, -1.0, 0.0})
        with([&](auto &q) { q.original_positions = v; }, "original_positions");
    for (double v : {nan, inf, 1.0, 0.0})
        with([&](auto &q) { q.beta_fast = v; }, "beta_fast");
    for (double v : {nan, inf, -1.0})
        with([&](auto &q) { q.attention_factor = v; }, "attention_factor");
    with([&](auto &q) { q.scaling = LORA_ROTARY_SCALE_BANDED; q.high_factor = nan; }, "high_factor");
    expect(lora_rotary_init(nullptr, &p), bad, "out NULL");
    expect(lora_rotary_init(&rot, nullptr), bad, "params NULL");

    const void *xs[1] = {nullptr};
    void *ys[1] = {nullptr};
    int32_t mods[1] = {0};
    const float scale = 1.f;
    expect(lora_base_load(nullptr, 0, &scale, &scale, nullptr, 128, nullptr), bad, "base_load: ctx NULL");
    expect(lora_base(nullptr, nullptr, nullptr, nullptr, 1, 0, nullptr), bad, "base: ctx NULL");
    expect(lora_base_group(nullptr, 1, mods, xs, xs, ys, 1, nullptr), bad, "base_group: ctx NULL");
    expect(lora_base_gated(nullptr, 0, 1, nullptr, nullptr, nullptr, nullptr, 1, 0, nullptr), bad,
           "base_gated: ctx NULL");
    expect(lora_rotary_group(nullptr, &rot, 1, mods, xs, ys, nullptr, 1, nullptr), bad,
           "rotary_group: ctx NULL");
    std::printf("failures: %d\n", failures);
    return failures != 0;
}
