// layer_load_check.cpp -- drives lora_base_load under AddressSanitizer and
// UndefinedBehaviorSanitizer without a GPU: the runtime's device calls are replaced
// by ones on host memory, each of which can be made to fail in its turn.  A load that
// fails must leave its module with the weight it had (before the first copy or pack is
// tried) or with none (from there on), never with a mixture.  Built and run by
// tests/test_layer_sanitizers_load.py.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "lora_mi355x.h"
#include "../../lora_adapter_application_amd/csrc/lora_layer.h"

static int failures = 0;
static int countdown = 0;      // the call that fails, counted from 1; 0: none
static int tried = 0;          // copies and packs of the present load
static bool fails() { return countdown > 0 && --countdown == 0; }

extern "C" {
hipError_t hipGetDeviceCount(int *n) { *n = 1; return hipSuccess; }
hipError_t hipGetDevice(int *d) { *d = 0; return hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipMalloc(void **p, size_t n)
{
    if (fails())
        return hipErrorOutOfMemory;
    *p = std::malloc(n);
    return *p ? hipSuccess : hipErrorOutOfMemory;
}
hipError_t hipFree(void *p) { std::free(p); return hipSuccess; }
hipError_t hipMemsetAsync(void *p, int v, size_t n, hipStream_t) { std::memset(p, v, n); return hipSuccess; }
hipError_t hipMemcpyAsync(void *d, const void *s, size_t n, hipMemcpyKind, hipStream_t)
{
    ++tried;
    if (fails())
        return hipErrorUnknown;
    std::memcpy(d, s, n);
    return hipSuccess;
}
hipError_t hipStreamCreateWithFlags(hipStream_t *s, unsigned) { *s = (hipStream_t)0x100; return hipSuccess; }
hipError_t hipStreamDestroy(hipStream_t) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipStreamQuery(hipStream_t) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus *c)
{
    *c = hipStreamCaptureStatusNone;
    return hipSuccess;
}
hipError_t hipStreamWaitEvent(hipStream_t, hipEvent_t, unsigned) { return fails() ? hipErrorUnknown : hipSuccess; }
hipError_t hipEventCreateWithFlags(hipEvent_t *e, unsigned)
{
    if (fails())
        return hipErrorOutOfMemory;
    *e = (hipEvent_t)0x200;
    return hipSuccess;
}
hipError_t hipEventDestroy(hipEvent_t) { return hipSuccess; }
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return fails() ? hipErrorUnknown : hipSuccess; }
hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }
// odd addresses stand for pinned host memory, which is staged; the rest for the device's
hipError_t hipPointerGetAttributes(hipPointerAttribute_t *a, const void *p)
{
    std::memset(a, 0, sizeof *a);
    a->type = ((uintptr_t)p & 1) ? hipMemoryTypeHost : hipMemoryTypeDevice;
    return hipSuccess;
}
}

static int launched_spb;
static const void *launched_bias, *launched_sc;

namespace lora {
static hipError_t reached() { return hipErrorNotSupported; }
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
hipError_t scratch_address(int, void **p) { *p = nullptr; return hipSuccess; }
hipError_t xcd_dispatch_check(int, hipStream_t, bool *ok) { *ok = false; return hipSuccess; }
hipError_t launch_base_pack(bool, const BasePackArgs &a, hipStream_t)
{
    ++tried;
    if (fails())
        return hipErrorLaunchFailure;
    // the last bytes of every source and destination are there
    const int64_t kb = (a.d_in + kBaseK - 1) / kBaseK, nb = (a.rows + kBaseCols - 1) / kBaseCols;
    volatile uint8_t sink = a.q[(int64_t)a.rows * a.d_in / 2 - 1];
    sink = (uint8_t)a.scale[(int64_t)a.rows * a.groups - 1];
    if (a.zero)
        sink = a.zero[(int64_t)a.rows * a.groups - 1];
    (void)sink;
    a.q_out[nb * kb * 256 - 1] = 1;
    ((uint32_t *)a.sc_out)[nb * kb * kBaseCols * a.spb - 1] = 1;
    *a.has_zero = a.zero != nullptr;
    return hipSuccess;
}
hipError_t launch_base(bool, bool, int spb, const BaseArgs &a, hipStream_t)
{
    launched_spb = spb;
    launched_bias = a.m[0].bias;
    launched_sc = a.m[0].sc;
    return hipSuccess;
}
hipError_t launch_rotary(bool, bool, const RotaryArgs &, hipStream_t) { return reached(); }
}  // namespace lora

#define CHECK(cond)                                                             \
    do {                                                                        \
        if (!(cond)) {                                                          \
            std::printf("FAIL line %d: %s (failing call %d)\n", __LINE__, #cond, k); \
            ++failures;                                                         \
        }                                                                       \
    } while (0)

int main()
{
    for (const int d_in : {8, 264})
        for (const int host : {0, 1}) {
            const int d_out = 72;
            const lora_module_shape shapes[1] = {{d_in, d_out}};
            // sources at even (device) or odd (pinned) addresses
            std::vector<uint8_t> q(d_out * d_in / 2 + 16), zero(d_out * 16 + 16);
            std::vector<uint16_t> bias(d_out + 16);
            std::vector<float> scale(d_out * 16 + 16);
            const uint8_t *pq = q.data() + host, *pz = zero.data() + host;
            const float *ps = scale.data();
            bool done = false;
            for (int k = 1; !done; ++k) {
                lora_ctx *ctx = nullptr;
                countdown = 0;
                CHECK(lora_slots_create(&ctx, 1, 1, shapes, 1, LORA_BF16, 8, 0) == LORA_OK);
                std::vector<uint16_t> x(8 * d_in), y(8 * d_out);
                CHECK(lora_base_load(ctx, 0, pq, ps, pz, 128, nullptr) == LORA_OK);
                CHECK(lora_base(ctx, x.data(), nullptr, y.data(), 8, 0, nullptr) == LORA_OK);
                CHECK(launched_spb == 1 && !launched_bias);
                const void *sc = launched_sc;
                // groups of 32 and a bias: every allocation that a reload can make
                tried = 0;
                countdown = k;
                const int rc = lora_base_load(ctx, 0, pq, ps, pz, 32, bias.data());
                done = countdown > 0;          // no call was left to fail
                countdown = 0;
                const int run = lora_base(ctx, x.data(), nullptr, y.data(), 8, 0, nullptr);
                if (done) {
                    CHECK(rc == LORA_OK && run == LORA_OK);
                    CHECK(launched_spb == 4 && launched_bias && launched_sc != sc);
                } else {
                    CHECK(rc != LORA_OK);
                    if (tried) {
                        CHECK(run == LORA_ERR_INVALID_ARGUMENT);
                        CHECK(std::strstr(lora_last_error(ctx), "no base weight"));
                    } else {
                        CHECK(run == LORA_OK && launched_spb == 1 && !launched_bias && launched_sc == sc);
                    }
                    // the next load makes the module whole
                    CHECK(lora_base_load(ctx, 0, pq, ps, pz, 32, bias.data()) == LORA_OK);
                    CHECK(lora_base(ctx, x.data(), nullptr, y.data(), 8, 0, nullptr) == LORA_OK);
                    CHECK(launched_spb == 4 && launched_bias);
                }
                lora_slots_destroy(ctx);
                if (k > 200) {
                    std::printf("FAIL no end\n");
                    return 1;
                }
            }
        }
    std::printf("failures: %d\n", failures);
    return failures != 0;
}
