// lora_ctx.h -- the ctx behind the C ABI and the host helpers that the runtime's
// source files share.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <memory>
#include <string>
#include <vector>

#include "../../include/lora_mi355x.h"
#include "lora_attend.h"
#include "lora_internal.h"
#include "lora_layer.h"

namespace lora {

struct StreamState {
    hipStream_t stream;
    uint64_t waited_gen;    // load generation this stream has waited for
    bool used_since_load;   // launched on since the last load
    bool since_fence;       // launched on since the side stream last waited for it
    hipEvent_t tail;        // recorded at load time to fence the stream's tail
    bool base_since_load;   // launched a base product since the last base load
    uint64_t base_waited;   // base-load generation this stream has waited for
};

struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev)
    {
        if (hipGetDevice(&prev) != hipSuccess)
            prev = -1;
        if (prev != dev)
            ok = hipSetDevice(dev) == hipSuccess;
    }
    ~DeviceGuard()
    {
        if (prev >= 0)
            (void)hipSetDevice(prev);
    }
};

inline int round_up(int v, int m) { return (v + m - 1) / m * m; }
inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Where one batch's plan and h partials live: the ctx's own allocation, or the
// library's static scratch array (lora_apply_group_noalloc).
struct Workspace {
    PlanBuffers plan{};
    float *hpart = nullptr;
    int hbuf_rows = 0;       // rows of one group member's block of h partials
    uint32_t *sync = nullptr;   // fused decode counts [max_tiles][kSyncWordsPerTile], kept at zero
                                // between launches (null: no fused launches on this workspace)
};

// The plan of the current batch, and the module list of the last shrink (which
// the expand must repeat).
struct BatchState {
    bool hinted = false;     // the batch declared its slots (lora_plan_prepare_slots)
    int plan_mode = kPlanTiles;   // PlanMode of the next bf16 launch on this plan
    int tile_cap = kTileTokens;   // tokens per tile of the plan
    const int32_t *idx = nullptr;
    int32_t T = 0;
    int last_n = 0;
    int last_modules[kMaxGroup] = {};
    int last_splits[kMaxGroup] = {};
    const void *last_x[kMaxGroup] = {};   // inputs of the last shrink (saved modules read them)
};

// The prepared batch of lora_attend and the workspace that its plan and parts are cut from.  Plans of
// captured prepares have a place of their own: a graph that is replayed writes its plan again, and an
// eager one has to stay.  Parts are of one lora_attend call, and all calls share their place.
struct AttendState {
    bool prepared = false;
    AttendBatch batch{};
    int head_dim = 0;
    unsigned long long capture = 0;      // the capture its plan was prepared in, or 0
    char *plans = nullptr;               // [2][plan_bytes]: eager, captured
    char *parts_base = nullptr;
    size_t plan_bytes = 0, parts_bytes = 0;
    float *parts[2] = {}, *sums[2] = {};
};

}  // namespace lora

// A paged cache; its memory is one of the ctx's allocations.
struct lora_cache {
    lora::CacheView view{};
};

struct lora_ctx {
    int device = 0;
    lora_dtype dtype = LORA_BF16;
    int S = 0, R = 0, R_pad = 0, n_modules = 0, max_tokens = 0, elem = 2;
    std::vector<lora_module_shape> shapes;
    std::vector<void *> A, Bi;
    std::vector<void *> bias;                // per module: [max_loras][d_out], ctx dtype
    std::vector<float *> dora;               // per module: [max_loras][d_out]
    std::vector<uint8_t> slot_flags;         // [S]: kSlotBias | kSlotDora
    // saved modules (lora_slot_load_saved): per module a pool [S][d_out][d_in] and
    // its biases [S][d_out], allocated at the module's first saved load
    std::vector<void *> saved_W, saved_bias;
    std::vector<uint8_t> saved_host;         // [n_modules][S]: 1 = the slot saves the module
    std::vector<uint8_t> saved_bias_host;    // [n_modules][S]: ... with a bias
    std::vector<int64_t> strideA, strideB;   // per-slot element strides
    std::vector<int32_t> rank_host;          // [n_modules][S]: r if the slot's adapter targets m
    std::vector<int32_t> slot_rank;          // [S]: rank of the adapter in the slot (0 = empty)
    std::vector<float> scale_host;
    void *stage = nullptr;                   // A^T and B staging for the modules of one load
    int64_t stage_elems = 0;
    lora::Workspace ws;                            // the ctx's plan buffers and h partials
    int max_tiles = 0;
    void *scratch = nullptr;                 // this device's static scratch array (no-alloc calls)
    bool xcd_local = false;                  // workgroups equal mod 8 share an XCD (fused decode hand-over in L2)
    hipStream_t side = nullptr;
    hipEvent_t load_done = nullptr;
    uint64_t load_gen = 0;
    uint64_t synced_gen = 0;                 // loads the host has seen complete (lora_sync_loads)
    // slots the prepared plan reads (lora_plan_prepare_slots, bs.hinted); else every slot
    std::vector<uint8_t> hint;               // [S]
    // per slot, the number of the last use event recorded after a launch of a
    // declared plan that reads it (0: none since the slot's last load)
    std::vector<uint64_t> last_use;          // [S]
    static constexpr int kUseEvents = 64;    // ring; a reused entry only waits longer
    hipEvent_t use_ev[kUseEvents] = {};
    uint64_t use_seq = 0;
    std::vector<lora::StreamState> streams;
    // plan state of the ctx's workspace; an inline plan is computed by the
    // first shrink launch itself
    bool plan_valid = false, plan_prepared = false;
    lora::BatchState bs;
    uint64_t slot_epoch = 0, shrink_epoch = 0;   // loads + clears, and their count at the last shrink
    lora_stats stats{};
    // kernel timing (lora_profile_begin / lora_profile_end)
    bool profiling = false;
    std::vector<lora::LaunchTiming> prof_events;
    std::vector<int> prof_kind;
    size_t prof_used = 0, prof_cap = 0;
    int64_t prof_untimed = 0;
    std::string last_error;
    std::vector<lora::BasePack> base;        // per module its 4-bit base weight (lora_base_load)
    hipEvent_t base_done = nullptr;          // the last base load; slot loads have load_done
    uint64_t base_gen = 0, base_synced = 0;  // base loads, and those the host has seen complete
    std::vector<std::unique_ptr<lora_cache>> caches;
    lora::AttendState attend;
    std::vector<void *> allocations;
    uint32_t flags_host = 0;                 // lora_get_device_flags' copy of the sticky word
};

namespace lora {

// Record a formatted message as the ctx's last error (ctx NULL: the thread's,
// which lora_last_error(NULL) returns) and give the status back.
int fail(lora_ctx *c, int status, const char *fmt, ...);
int hip_fail(lora_ctx *c, hipError_t e, const char *what);

#define HIP_TRY(ctx, expr)                                   \
    do {                                                     \
        hipError_t e_ = (expr);                              \
        if (e_ != hipSuccess)                                \
            return hip_fail((ctx), e_, #expr);               \
    } while (0)

// The ctx's record of stream s (made at its first launch there), or NULL.
StreamState *stream_state(lora_ctx *c, hipStream_t s);
// Whether s is being captured into a graph.
bool stream_capturing(hipStream_t s);

// A load source must be pinned host, device or managed memory.  *in_place:
// the finalize kernel on `device` may read it at its own address (memory of
// that device, managed memory, or pinned host memory mapped at its host
// address) and it is 16-byte aligned; otherwise it is staged by a copy.
int check_source(const void *p, int device, bool *in_place = nullptr);

inline int check_ctx(lora_ctx *c) { return c ? LORA_OK : LORA_ERR_INVALID_ARGUMENT; }

// Argument checks of the grouped calls.
int check_group(lora_ctx *c, int32_t n, const int32_t *modules);
int check_ptrs(lora_ctx *c, int32_t n, const void *const *p, const char *what, bool distinct);

}  // namespace lora
