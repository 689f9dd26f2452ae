// lora_attend.hip -- gfx950 kernels of attention over the paged cache.
//
//     o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q . k_t - m),
//
// over the tokens t that a row sees: its prefix's and its own request's up to itself.  Both
// products run on the matrix cores with the tokens as rows, S^T = K Q^T and O^T = V^T P^T: the
// result layout of the first is the operand layout of the second (a lane keeps 8 tokens of one
// row), so weights go from product to product in registers, and the cache's order makes every
// operand one contiguous read.  The running maximum m is raised only when a score passes it by
// 2^8, which keeps weights far inside fp32 and skips most rescalings; sums are fp32.  The second
// product of a bf16 ctx takes weights as two bf16 in narrow tiles, off by 2^-15 of a weight at most (2^-16
// over codes), and as one in wide tiles, off by 2^-8 (as large an error as that of the rounded result);
// the sum is that of the unrounded ones.  The relative 2-norm errors of results are 0.0016 to 0.0017 and
// 0.0023 to 0.0024.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "lora_attend.h"
#include "lora_dma.h"

namespace lora {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;

constexpr float kRaise = 8.f;        // a maximum is raised when a score passes it by 2^8
#define kNone (-__builtin_inff())

// ---------------------------------------------------------------------------
// plan: one workgroup turns the batch's lengths into the two lists of tiles
//
// 256 to 512 requests take 9 to 11 us, latency throughout: lengths, counts, sums over the workgroup,
// tiles, the search for each worker's first tile, a barrier between each.  One workgroup, because
// several would have to wait for each other's sums, about a launch each; sums in LDS and registers,
// because a barrier that also waits for memory costs 1 us.

constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
constexpr int kPlanUnits = 2048;     // tiles of a list whose first units stand in LDS for the workers' search
constexpr int kPlanSeqs = 2048;      // requests whose listed tokens stand in LDS
constexpr int kPlanEach = 4;         // tiles a thread writes by itself; a wave writes those of larger entities

// What an entity adds to the lists.  Where requests, or prefixes, claim more tokens than there are
// these sums may wrap; such a batch is found by sums of 64 bits and gets no work.
struct PlanCount { int32_t v[6]; };  // tiles, kept tiles, units of the two lists

// Inclusive sums over the lanes of a wave, and over each 16 of them.
template <int CTRL, int ROWS>
__device__ __forceinline__ int32_t from_lane(int32_t v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int32_t row_scan(int32_t v)
{
    v += from_lane<0x111, 0xf>(v);       // the lane 1 before, in its row of 16
    v += from_lane<0x112, 0xf>(v);
    v += from_lane<0x114, 0xf>(v);
    v += from_lane<0x118, 0xf>(v);
    return v;
}
__device__ __forceinline__ int32_t wave_scan(int32_t v)
{
    v = row_scan(v);
    v += from_lane<0x142, 0xa>(v);       // the last of the row before, to rows 1 and 3
    v += from_lane<0x143, 0xc>(v);       // lane 31, to rows 2 and 3
    return v;
}

// A barrier behind which the workgroup sees its writes to LDS; unlike __syncthreads it does not wait
// for writes to memory, about 1 us each.
__device__ __forceinline__ void lds_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__global__ __launch_bounds__(kPlanThreads) void attend_plan_kernel(AttendBatch b)
{
    constexpr int threads = kPlanThreads, waves = kPlanWaves;
    __shared__ int32_t wave_sum[7][kPlanWaves];
    __shared__ int32_t unit0[2][kPlanUnits];
    __shared__ int32_t bounds[LORA_ATTEND_MAX_PREFIXES + 1], pre_len[LORA_ATTEND_MAX_PREFIXES];
    __shared__ AttendEntity large[kPlanThreads];
    __shared__ unsigned long long large_units[kPlanThreads];
    __shared__ int32_t large_at[kPlanThreads][4], n_large;
    __shared__ int32_t listed_before[kPlanSeqs + 1];
    __shared__ unsigned long long sums[3];   // new tokens, tokens listed for prefixes, units
    __shared__ int bad_any;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the first requests' words are on their way before the first barrier
    Request words{};
    if (tid < b.n_seqs)
        words = request_words(b, tid);
    const bool small = b.n_seqs <= kPlanSeqs;
    const int entities = b.n_seqs + b.n_prefixes;
    // (no pointer to either: a read through that would wait for every write under way)
    auto before = [&](int i) {
        if (small)
            return listed_before[i];
        return b.list_before[i];
    };
    if (tid < 3)
        sums[tid] = 0;
    if (!tid) {
        bad_any = 0;
        n_large = 0;
    }
    AttendBatch c = b;                   // with the prefixes' bounds and lengths from LDS
    c.prefix_seqs = bounds;
    c.prefix_lengths = pre_len;
    if (b.n_prefixes) {
        for (int i = tid; i <= b.n_prefixes; i += threads)
            bounds[i] = b.prefix_seqs[i];
        for (int i = tid; i < b.n_prefixes; i += threads)
            pre_len[i] = b.prefix_lengths[i];
    }
    lds_sync();
    bool bad = false;
    AttendEntity e{};
    // sum over the workgroup of one value a thread: those before the thread's, and all
    auto sum_before = [&](int k, int32_t v, int32_t &all) {
        const int32_t incl = row_scan((lane & 15) < waves ? wave_sum[k][lane & 15] : 0);
        all = __builtin_amdgcn_readlane(incl, 15);
        return (wave ? __builtin_amdgcn_readlane(incl, wave - 1) : 0) + v;
    };

    // the tokens of requests that share a prefix, request by request
    int32_t n_listed = 0;
    if (b.n_prefixes) {
        for (int from = 0; from < b.n_seqs; from += threads) {
            const int i = from + tid;
            int32_t own = 0;
            if (from + wave * 64 < b.n_seqs) {                 // waves without requests only keep the barriers
                if (i < b.n_seqs) {
                    e = request_of(c, i, from ? request_words(b, i) : words, &bad);
                    own = e.listed;
                }
                own = wave_scan(own);
                if (lane == 63)
                    wave_sum[0][wave] = own;
            } else if (!lane) {
                wave_sum[0][wave] = 0;
            }
            lds_sync();
            int32_t all;
            const int32_t at = n_listed + sum_before(0, own, all) - e.listed;
            if (i < b.n_seqs) {
                b.list_before[i] = at;
                if (small)
                    listed_before[i] = at;
                for (int j = 0; j < e.listed; ++j)
                    if ((uint32_t)(at + j) < (uint32_t)b.n_tokens)
                        b.listed[at + j] = e.token0 + j;
            }
            n_listed += all;
            lds_sync();
        }
        if (!tid) {
            if (small)
                listed_before[b.n_seqs] = n_listed;
            else
                b.list_before[b.n_seqs] = n_listed;
        }
        if (small)
            lds_sync();
        else
            __syncthreads();
    }

    // the tiles of requests and of prefixes
    auto entity_of = [&](int i, const Request &r, bool *flag) {
        if (i < b.n_seqs)
            return request_of(c, i, r, flag);
        const int p = i - b.n_seqs, s0 = c.prefix_seqs[p], s1 = c.prefix_seqs[p + 1];
        *flag |= s0 < 0 || s1 < s0 || s1 > b.n_seqs;
        const int lo = clamp_to(s0, 0, b.n_seqs), hi = clamp_to(s1, lo, b.n_seqs);
        const int l0 = before(lo);
        return prefix_of_batch(c, p, l0, before(hi) - l0, flag);
    };
    int32_t base[6] = {};
    unsigned long long sum[3] = {};
    for (int from = 0; from < entities; from += threads) {
        const int i = from + tid;
        PlanCount n{}, at{};
        const bool any = from + wave * 64 < entities;
        int mine = -1;                                         // the thread's number among the large
        if (any) {
            if (i >= entities)
                e = AttendEntity{};
            else if (from || i >= b.n_seqs || !b.n_prefixes || b.n_seqs > threads)   // else as found above
                e = entity_of(i, from && i < b.n_seqs ? request_words(b, i) : words, &bad);
            if (e.tiles > kPlanEach) {
                mine = atomicAdd(&n_large, 1);                 // their order changes no place
                large[mine] = e;
            }
        }
        lds_sync();
        const int count = n_large;
        if (count) {                                           // their units, a wave each
            for (int k = wave; k < count; k += waves) {
                unsigned long long units = 0;
                for (int j = lane; j < large[k].tiles; j += 64)
                    units += tile_of(b, large[k], j, 0).units;
                for (int d = 1; d < 64; d <<= 1)
                    units += __shfl_xor(units, d);
                if (!lane)
                    large_units[k] = units;
            }
            lds_sync();
        }
        if (any) {
            unsigned long long units = 0;
            if (mine >= 0)
                units = large_units[mine];
            else
                for (int j = 0; j < e.tiles; ++j)
                    units += tile_of(b, e, j, 0).units;
            sum[0] += e.shared ? 0 : e.q_len;
            sum[1] += e.shared ? over_group(b, e.rows) : 0;
            sum[2] += units;
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                n.v[l] = e.list == l ? e.tiles : 0;
                n.v[2 + l] = e.list == l && e.keeps ? e.tiles : 0;
                n.v[4 + l] = e.list == l ? (int32_t)units : 0;
            }
#pragma unroll
            for (int k = 0; k < 6; ++k) {
                const int32_t incl = wave_scan(n.v[k]);
                if (lane == 63)
                    wave_sum[k][wave] = incl;
                at.v[k] = base[k] + incl - n.v[k];
            }
        } else if (lane < 6) {
            wave_sum[lane][wave] = 0;
        }
        lds_sync();
#pragma unroll
        for (int k = 0; k < 6; ++k) {
            int32_t all;
            at.v[k] = sum_before(k, at.v[k], all);
            base[k] += all;
        }
        if (any && i < entities) {
            const int l = e.list, tile = l ? at.v[1] : at.v[0];
            const int kept = l ? at.v[3] : at.v[2], u0 = l ? at.v[5] : at.v[4];
            const int list0 = e.prefix >= 0 ? before(i) : 0;
            if (i >= b.n_seqs)
                b.prefix_tile[i - b.n_seqs] = PrefixTile{l, tile};
            if (mine >= 0) {
                large_at[mine][0] = tile;
                large_at[mine][1] = kept;
                large_at[mine][2] = u0;
                large_at[mine][3] = list0;
            } else {
                int u = u0;
                for (int j = 0; j < e.tiles && (uint32_t)(tile + j) < (uint32_t)b.cap[l]; ++j) {
                    AttendTile t = tile_of(b, e, j, list0);
                    t.kept = e.keeps ? kept + j : -1;
                    t.unit0 = u;
                    u += t.units;
                    b.tiles[l][tile + j] = t;
                    if (tile + j < kPlanUnits)
                        unit0[l][tile + j] = t.unit0;
                }
            }
        }
        if (!count)
            continue;
        lds_sync();
        for (int k = wave; k < count; k += waves) {
            const int tile = large_at[k][0], kept = large_at[k][1];
            const AttendEntity g = large[k];
            int u = large_at[k][2];
            for (int j0 = 0; j0 < g.tiles; j0 += 64) {
                const int j = j0 + lane;
                AttendTile t{};
                if (j < g.tiles)
                    t = tile_of(b, g, j, large_at[k][3]);
                const int32_t incl = wave_scan(t.units);
                t.kept = g.keeps ? kept + j : -1;
                t.unit0 = u + incl - t.units;
                u += __builtin_amdgcn_readlane(incl, 63);
                if (j < g.tiles && (uint32_t)(tile + j) < (uint32_t)b.cap[g.list]) {
                    b.tiles[g.list][tile + j] = t;
                    if (tile + j < kPlanUnits)
                        unit0[g.list][tile + j] = t.unit0;
                }
            }
        }
        lds_sync();
        if (!tid)
            n_large = 0;
        lds_sync();
    }
    if (bad)
        bad_any = 1;
    if (base[0] > kPlanUnits || base[1] > kPlanUnits)
        __syncthreads();                                       // first units that the search reads from memory
    else
        lds_sync();
    // A batch that claims tokens twice gets no work; one that is only out of order, the work that its
    // clamped values name.  Arrays in order claim none twice, and what they name fits.
    bool none = false;
    if (bad_any || !b.units_fit) {
#pragma unroll 1
        for (int k = 0; k < 3; ++k) {                          // whole numbers: their order changes nothing
            const unsigned long long v = k == 0 ? sum[0] : k == 1 ? sum[1] : sum[2];
            const uint32_t lo = wave_scan((int32_t)(v & 0xffffff)), hi = wave_scan((int32_t)(v >> 24));
            if (lane == 63 && (lo | hi))
                atomicAdd(&sums[k], ((unsigned long long)hi << 24) + lo);
        }
        lds_sync();
        none = !attend_fits(b, sums[0], sums[1], sums[2], base);
    }
    const int l = wave >= kPlanWaves / 2;                      // half of the threads for each list
    AttendList out{none ? 0 : l ? base[1] : base[0], none ? 0 : l ? base[5] : base[4], none ? 0 : l ? base[3] : base[2], 1};
    const int workers = l ? b.workers[1] : b.workers[0];
    const int64_t all = (int64_t)out.units * b.kv_heads;
    out.run = all ? worker_run(all, workers) : 1;
    if (tid == l * (kPlanThreads / 2))
        b.plan->list[l] = out;
    for (int w = tid & (kPlanThreads / 2 - 1); w < workers; w += kPlanThreads / 2) {
        const int64_t u = (int64_t)w * out.run;
        if (u >= all)
            break;
        const int32_t want = (int32_t)(u >> 32 ? u % out.units : (uint32_t)u % (uint32_t)out.units);
        int lo = 0, hi = out.tiles - 1;
        auto search = [&](auto &&first_unit) {
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (first_unit(mid) <= want)
                    lo = mid;
                else
                    hi = mid - 1;
            }
        };
        if (out.tiles <= kPlanUnits)
            search([&](int k) { return unit0[l][k]; });
        else
            search([&](int k) { return b.tiles[l][k].unit0; });
        b.start[l][w] = lo;
    }
    if (!tid) {
        b.plan->bad = none;
        if (none || bad_any)
            atomicOr(b.flags, LORA_FLAG_ATTEND_BATCH);
    }
}

// ---------------------------------------------------------------------------
// elements

template <typename T> struct Frag;                       // 8 inputs of a matrix instruction's lane
template <> struct Frag<uint16_t> { bf16x8 v; };
template <> struct Frag<float> { float v[8]; };

__device__ __forceinline__ f32x4 mma(const Frag<uint16_t> &a, const Frag<uint16_t> &b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(const Frag<uint16_t> &a, const Frag<uint16_t> &b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float> &a, const Frag<float> &b, f32x4 c)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ Frag<uint16_t> to_frag(const float *p, uint16_t)
{
    Frag<uint16_t> f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f.v[j] = (__bf16)p[j];
    return f;
}
__device__ __forceinline__ Frag<float> to_frag(const float *p, float)
{
    Frag<float> f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f.v[j] = p[j];
    return f;
}

// 8 elements as the cache holds them, and as a matrix instruction takes them.  Codes are
// exact in bf16 (4 and 8 significant bits).
template <typename T, int KIND> struct Held;
template <> struct Held<uint16_t, kCacheNative> { uint4 r; };
template <> struct Held<float, kCacheNative> { float4 r[2]; };
template <typename T> struct Held<T, kCacheFp8> { uint2 r; };
template <typename T> struct Held<T, kCacheInt8> { uint2 r; };

template <typename T, int KIND>
__device__ __forceinline__ Held<T, KIND> held_load(const char *base, int unit)
{
    return *(const Held<T, KIND> *)(base + (int64_t)unit * sizeof(Held<T, KIND>));
}

__device__ __forceinline__ void fp8_values(uint2 r, float *v)
{
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int x = w ? r.y : r.x;
        v[4 * w + 0] = __builtin_amdgcn_cvt_f32_fp8(x, 0);
        v[4 * w + 1] = __builtin_amdgcn_cvt_f32_fp8(x, 1);
        v[4 * w + 2] = __builtin_amdgcn_cvt_f32_fp8(x, 2);
        v[4 * w + 3] = __builtin_amdgcn_cvt_f32_fp8(x, 3);
    }
}
__device__ __forceinline__ void int8_values(uint2 r, float *v)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = (float)(int8_t)((j < 4 ? r.x : r.y) >> (8 * (j & 3)));
}

__device__ __forceinline__ Frag<uint16_t> frag_of(const Held<uint16_t, kCacheNative> &h)
{
    return {__builtin_bit_cast(bf16x8, h.r)};
}
__device__ __forceinline__ Frag<float> frag_of(const Held<float, kCacheNative> &h)
{
    return {{h.r[0].x, h.r[0].y, h.r[0].z, h.r[0].w, h.r[1].x, h.r[1].y, h.r[1].z, h.r[1].w}};
}
__device__ __forceinline__ Frag<float> frag_of(const Held<float, kCacheFp8> &h)
{
    float v[8];
    fp8_values(h.r, v);
    return to_frag(v, float());
}
__device__ __forceinline__ Frag<uint16_t> frag_of(const Held<uint16_t, kCacheFp8> &h)
{
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    Frag<uint16_t> f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const bf16x2 v = w & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w < 2 ? h.r.x : h.r.y, 1.f, true)
                               : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w < 2 ? h.r.x : h.r.y, 1.f, false);
        f.v[2 * w] = v[0];
        f.v[2 * w + 1] = v[1];
    }
    return f;
}
template <typename T>
__device__ __forceinline__ Frag<T> frag_of(const Held<T, kCacheInt8> &h)
{
    float v[8];
    int8_values(h.r, v);
    return to_frag(v, T());
}

// Elements from `keep` on become zero.
template <typename T>
__device__ __forceinline__ void cut(Frag<T> &f, int keep)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j >= keep)
            f.v[j] = 0;
}

template <typename T> struct Io;
template <> struct Io<uint16_t> {
    static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t put(float f)
    {
        __bf16 h = (__bf16)f;
        return __builtin_bit_cast(uint16_t, h);
    }
};
template <> struct Io<float> {
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float f) { return f; }
};

template <typename T, int N> struct alignas(sizeof(T) * N) Pack { T v[N]; };

// Four results of a row from dim d on; dims past head_dim are padding (head_dim is a multiple of 8).
template <typename T>
__device__ __forceinline__ void put4(T *y, const float *v, bool vec)
{
    if (vec) {
        Pack<T, 4> p;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p.v[i] = Io<T>::put(v[i]);
        *(Pack<T, 4> *)y = p;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = Io<T>::put(v[i]);
    }
}

// 8 elements of a q row
template <typename T>
__device__ __forceinline__ Frag<T> q_frag(const T *q, bool vec)
{
    Frag<T> f;
    if (vec) {
        f = __builtin_bit_cast(Frag<T>, *(const Pack<T, 8> *)q);
    } else {
        Pack<T, 8> p;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p.v[j] = q[j];
        f = __builtin_bit_cast(Frag<T>, p);
    }
    return f;
}

__device__ __forceinline__ int row_token(const AttendBatch &b, const AttendTile &t, int r)
{
    const int at = t.token0 + over_group(b, r);
    return t.shared ? b.listed[at] : at;
}

// Plan words that a whole workgroup works by, in scalar registers.
template <typename P>
__device__ __forceinline__ P scalar(const P *p)
{
    P r;
    const int32_t *from = (const int32_t *)p;
    int32_t *to = (int32_t *)&r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(P) / 4); ++i)
        to[i] = __builtin_amdgcn_readfirstlane(from[i]);
    return r;
}

__device__ __forceinline__ const char *scalar_address(const char *p)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)(uint64_t)p);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)p >> 32));
    return (const char *)((uint64_t)hi << 32 | lo);
}

// Workgroups of one XCD take neighbouring runs: tiles of one prefix or request, and so the pages
// they read, stay in one L2.
__device__ __forceinline__ int worker_of_block() { return (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3); }

__device__ __forceinline__ float fexp2(float x) { return __builtin_amdgcn_exp2f(x); }

// at / units: a key-value head.
__device__ __forceinline__ int div_small(int64_t at, int32_t units)
{
    return at >> 32 ? (int)(at / units) : (int)((uint32_t)at / (uint32_t)units);
}

// ---------------------------------------------------------------------------
// simple batches: a workgroup sums the requests' units itself, one a thread
//
// Saves the plan's launch, 9 us of what is 18 for a single token over 2047 others without it.

struct SimplePlan {
    int32_t len[kSimpleSeqs], unit0[kSimpleSeqs], sum[4];
};
__device__ __forceinline__ AttendList plan_simple(const AttendBatch &b, SimplePlan &p)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    bool bad = false;
    const int len = tid < b.n_seqs ? held_of(b.lengths[tid], b.max_pages, b.page_shift, &bad) : 0;
    if (bad && !blockIdx.x && !blockIdx.y)
        atomicOr(b.flags, LORA_FLAG_ATTEND_BATCH);
    const int units = tid < b.n_seqs ? simple_tile(tid, len, b.group, 0).units : 0;
    const int incl = wave_scan(units);
    if (lane == 63)
        p.sum[wave] = incl;
    lds_sync();
    int before = incl - units, all = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        before += k < wave ? p.sum[k] : 0;
        all += p.sum[k];
    }
    p.len[tid] = len;
    p.unit0[tid] = before;
    lds_sync();
    all = __builtin_amdgcn_readfirstlane(all);
    return {b.n_seqs, all, 0, worker_run((int64_t)all * b.kv_heads, b.workers[0])};
}
// The tile with unit u.
__device__ __forceinline__ int find_simple(const SimplePlan &p, int u, int tiles)
{
    int lo = 0, hi = tiles - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__builtin_amdgcn_readfirstlane(p.unit0[mid]) <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// ---------------------------------------------------------------------------
// narrow tiles: 16 rows, four waves on 32 tokens each of a unit of 128
//
// For rows so few that reading the cache is the work: 16 is the least that a matrix instruction takes,
// and the waves split the tokens, since all of them need the same few rows.  Operands go from memory
// to registers, no LDS between; the four waves' results meet in LDS once a tile.  Bytes bound it where
// there are enough: 256 requests of up to 2048 and 8 prefixes, fp8, 440 us (5.1 TB/s); one token over 2047,
// 12 us, one or two units a worker: the chain page, keys, scores, values, sums, part.  With heads in
// groups of 8 half of the 16 rows carry nothing and conversions of codes count too (512 requests,
// int8, 271 thousand tokens of 8 heads, 146 us, 3.9 TB/s).  Not kept: fetching the next block's keys ahead within the wave costs the
// registers of the other workgroups on the CU (494 to 620 us when it was tried), as do four
// workgroups a CU at 128 dims of codes (spills, +14%).

// The contribution of values that are infinite or NaN, for blocks of which rows see different
// tokens: a hidden token's weight is 0, and 0 times those is NaN.  Their places are taken out of
// the product (v becomes 0 there), and each row gets what the tokens that it sees bring.
template <typename T, typename Acc>
__device__ __forceinline__ void odd_values(Frag<T> &v, const Frag<T> &sees, Acc &o)
{
    bool any = false;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        any |= !(__builtin_fabsf((float)v.v[j]) < __builtin_inff());
    if (!__any(any))
        return;
    const float bring[3] = {__builtin_inff(), -__builtin_inff(), __builtin_nanf("")};
#pragma unroll 1
    for (int k = 0; k < 3; ++k) {
        Frag<T> where{};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = (float)v.v[j];
            where.v[j] = (k == 2 ? x != x : x == bring[k]) ? 1.f : 0.f;
        }
        const Acc seen = mma(where, sees, Acc{});
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Acc) / 4); ++i)
            if (seen[i] > 0)
                o[i] += bring[k];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (!(__builtin_fabsf((float)v.v[j]) < __builtin_inff()))
            v.v[j] = 0.f;
}

template <typename T, int KIND, int DP>
__global__ __launch_bounds__(256, kAttendPerCu(sizeof(T), KIND, DP)) void attend_narrow_kernel(AttendArgs a)
{
    constexpr int NS = DP / 32, ND = DP / 16, W = DP + 4;
    __shared__ float lds_o[4][kNarrowRows][W];
    __shared__ float lds_m[4][kNarrowRows], lds_l[4][kNarrowRows];
    __shared__ SimplePlan own;
    const AttendBatch &b = a.b;
    const int w = worker_of_block();
    AttendList list;
    int first = 0, bad = 0;
    if (b.simple) {
        list = plan_simple(b, own);
    } else {
        list = scalar(&b.plan->list[0]);
        first = scalar(b.start[0] + w);                      // stale if the worker has no work
        bad = scalar(&b.plan->bad);
    }
    const int64_t total = bad ? 0 : (int64_t)list.units * b.kv_heads;
    int64_t at = (int64_t)w * list.run;
    const int64_t end = at + list.run < total ? at + list.run : total;
    if (at >= end)
        return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const int heads = b.group * b.kv_heads, hd = a.c.head_dim;
    const bool vec = (((uintptr_t)a.q | (uintptr_t)a.y) & 15) == 0;
    int head = __builtin_amdgcn_readfirstlane(div_small(at, list.units));
    int x = b.simple ? find_simple(own, (int)(at - (int64_t)head * list.units), list.tiles) : first;

    for (; at < end; ++x) {
        if (x == list.tiles) {
            x = 0;
            ++head;
        }
        AttendTile t;
        if (b.simple)
            t = simple_tile(x, __builtin_amdgcn_readfirstlane(own.len[x]), b.group, __builtin_amdgcn_readfirstlane(own.unit0[x]));
        else
            t = scalar(b.tiles[0] + x);
        const int64_t base = (int64_t)head * list.units + t.unit0;
        const int u0 = (int)(at - base);
        const int u1 = (int)((end < base + t.units ? end : base + t.units) - base);

        const int row = t.row0 + n;
        const bool mine = n < t.rows;
        Frag<T> q[NS];
        {
            const int r = mine ? row : t.row0;
            const int token = row_token(b, t, r);
            const T *p = (const T *)a.q + ((int64_t)token * heads + head * b.group + (r - over_group(b, r) * b.group)) * hd;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int d = 32 * s + 8 * g;
                q[s] = Frag<T>{};
                if (mine && d < hd)
                    q[s] = q_frag<T>(p + d, vec);
            }
        }
        // tokens of the request's own pages that this lane's row sees, the fewest and the most of the tile
        const int per = t.shared ? 0 : t.len - t.q_len + 1;
        const int see = t.shared ? t.len : per + over_group(b, mine ? row : t.row0 + t.rows - 1);
        const int see_min = t.shared ? t.len : per + over_group(b, t.row0);
        const int see_max = t.shared ? t.len : per + over_group(b, t.row0 + t.rows - 1);
        const int pre_units = units_for(t.pre_len, kNarrowUnit);
        const int32_t *own_pages = t.shared ? b.prefix_pages + (int64_t)t.seq * b.prefix_max_pages
                                            : b.pages + (int64_t)t.seq * b.max_pages;
        const int32_t *pre_pages = t.pre_len ? b.prefix_pages + (int64_t)t.pre_seq * b.prefix_max_pages : nullptr;

        // Where the wave's blocks are: each lane holds the address of that of one unit, 64 at a time, so
        // that no load of keys waits for one of a page.  Blocks that no row sees have the cache's first page.
        bool lost = false;                                   // a page was not one of the cache's
        uint32_t far_lo = 0, far_hi = 0;
        int far0 = 0;
        auto look = [&](int u) __attribute__((always_inline)) {
            far0 = u;
            const int uu = u + lane;
            const bool in_pre = uu < pre_units;
            const int tok0 = (in_pre ? uu : uu - pre_units) * kNarrowUnit + wave * kBlock;
            int page = 0;
            if (uu < u1 && tok0 < (in_pre ? t.pre_len : see_max))
                page = (in_pre ? pre_pages : own_pages)[tok0 >> a.c.page_shift];
            const bool good = (uint32_t)page < (uint32_t)a.c.pages;
            lost |= __any(!good);
            const uint64_t p = (uint64_t)(a.c.base + cache_block(a.c, good ? page : 0, head,
                                                                 (tok0 >> 5) & ((1 << (a.c.page_shift - 5)) - 1)));
            far_lo = (uint32_t)p;
            far_hi = (uint32_t)(p >> 32);
        };

        f32x4 o[ND];
#pragma unroll
        for (int d = 0; d < ND; ++d)
            o[d] = f32x4{0, 0, 0, 0};
        float m = kNone, l = 0;
        // The wave's block of a unit; MASKED: some rows do not see all of its tokens.
        auto work = [&](auto masked, int u) __attribute__((always_inline)) {
            constexpr bool MASKED = decltype(masked)::value;
            if (u - far0 >= 64)
                look(u);
            const uint32_t lo = __builtin_amdgcn_readlane(far_lo, u - far0), hi = __builtin_amdgcn_readlane(far_hi, u - far0);
            const char *blk = (const char *)((uint64_t)hi << 32 | lo);
            int here = 0, most = 0;                          // tokens of the block that this row sees, that any of the tile does
            if constexpr (MASKED) {
                const bool in_pre = u < pre_units;
                const int tok0 = (in_pre ? u : u - pre_units) * kNarrowUnit + wave * kBlock;
                here = (in_pre ? t.pre_len : see) - tok0;
                most = (in_pre ? t.pre_len : see_max) - tok0;
                if (most <= 0)
                    return;
            }
            Held<T, KIND> kh[2][NS], vh[ND];
            const int km = 8 * (n >> 2) + (n & 3);
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    kh[c][s] = held_load<T, KIND>(blk, (4 * s + g) * kBlock + km + 4 * c);
            f32x4 ks[2], vs[2];                              // of codes: of tokens 8 g + 4 c + i
            if constexpr (KIND != kCacheNative)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    ks[c] = *(const f32x4 *)(blk + 2 * a.c.half + (8 * g + 4 * c) * 4);
                    vs[c] = *(const f32x4 *)(blk + 2 * a.c.half + (kBlock + 8 * g + 4 * c) * 4);
                }
#pragma unroll
            for (int d = 0; d < ND; ++d)
                vh[d] = held_load<T, KIND>(blk + a.c.half, g * DP + 16 * d + n);
            f32x4 st[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    st[c] = mma(frag_of(kh[c][s]), q[s], st[c]);
            // scores in powers of two; token 8 g + 4 c + i of the block
            float p[8];
            float top = kNone;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = st[c][i] * a.scale;
                    if constexpr (KIND != kCacheNative)
                        v *= ks[c][i];
                    if (MASKED && 8 * g + 4 * c + i >= here)
                        v = kNone;
                    p[4 * c + i] = v;
                    top = __builtin_fmaxf(top, v);
                }
            top = __builtin_fmaxf(top, __shfl_xor(top, 16));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            if (__any(top > m + kRaise)) {
                const float up = __builtin_fmaxf(m, top);
                const float f = up == kNone ? 1.f : fexp2(m - up);
                m = up;
                l *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    o[d] *= f;
            }
            const float off = m == kNone ? 0.f : m;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j] = fexp2(p[j] - off);
                l += p[j];
                if constexpr (KIND != kCacheNative)          // a hidden token's scale may be NaN
                    p[j] = MASKED && 8 * g + j >= here ? 0.f : p[j] * vs[j >> 2][j & 3];
            }
            // A bf16 ctx takes weights in two parts: loads bound this kernel and the second product costs
            // under 1%.  Of codes, which are finite, a part is rounded and the second is what that leaves, of either
            // sign.  Values as they are may be infinite: there the first part is cut off and the second has its
            // sign, at least 2^-40 of it and no less than bf16 holds, so that both products with an infinity agree.
            constexpr bool FINE = sizeof(T) == 2;
            float first[8], second[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                first[j] = p[j];
                if constexpr (FINE && KIND == kCacheNative)
                    first[j] = __uint_as_float(__float_as_uint(p[j]) & 0xffff0000u);
            }
            const Frag<T> pf = to_frag(first, T());
            Frag<T> rest{};
            if constexpr (FINE) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    second[j] = KIND == kCacheNative
                        ? __builtin_fmaxf(p[j] - first[j], __builtin_amdgcn_fmed3f(first[j], first[j] * 0x1p-40f, 0x1p-126f))
                        : p[j] - (float)pf.v[j];
                rest = to_frag(second, T());
            }
            Frag<T> sees{};
            if constexpr (MASKED && KIND == kCacheNative)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sees.v[j] = 8 * g + j < here ? 1.f : 0.f;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                Frag<T> v = frag_of(vh[d]);
                if constexpr (MASKED) {                      // what no row sees may hold anything
                    cut(v, most - 8 * g);
                    if constexpr (KIND == kCacheNative)
                        odd_values<T>(v, sees, o[d]);
                }
                o[d] = mma(v, pf, o[d]);
                if constexpr (FINE)
                    o[d] = mma(v, rest, o[d]);
            }
        };
        look(u0);
        // units before these have whole blocks of the wave's; rounded down, also below zero
        static_assert(kNarrowUnit == 128, "");
        const int pre_full = ((t.pre_len - (wave + 1) * kBlock) >> 7) + 1;
        const int own_full = pre_units + ((see_min - (wave + 1) * kBlock) >> 7) + 1;
        for (int u = u0; u < u1;) {
            const int full = u < pre_units ? pre_full : own_full;
            const int stop = full < u1 ? full : u1;
            for (; u < stop; ++u)
                work(std::false_type(), u);
            if (u < u1)
                work(std::true_type(), u++);
        }
        if (lost) {
            l = __builtin_nanf("");
            if (!lane)
                atomicOr(b.flags, LORA_FLAG_CACHE_PAGE);
        }

        // join the waves
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (g == 0) {
            lds_m[wave][n] = m;
            lds_l[wave][n] = l;
        }
        __syncthreads();
        {
            const float top = __builtin_fmaxf(__builtin_fmaxf(lds_m[0][n], lds_m[1][n]),
                                              __builtin_fmaxf(lds_m[2][n], lds_m[3][n]));
            const float f = m == kNone ? (l != l ? l : 0.f) : fexp2(m - top);
#pragma unroll
            for (int d = 0; d < ND; ++d)
                *(f32x4 *)&lds_o[wave][n][16 * d + 4 * g] = o[d] * f;
        }
        __syncthreads();
        const bool whole = t.kept < 0 && u0 == 0 && u1 == t.units;
        const int64_t slot = part_slot(list, b.workers[0], head, t, w);
        for (int i = threadIdx.x; i < t.rows * (DP / 4); i += 256) {
            const int r = i / (DP / 4), d = i % (DP / 4) * 4;
            float top = kNone, sum = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                top = __builtin_fmaxf(top, lds_m[k][r]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sum += lds_m[k][r] == kNone ? lds_l[k][r] : lds_l[k][r] * fexp2(lds_m[k][r] - top);
            f32x4 v = *(const f32x4 *)&lds_o[0][r][d];
#pragma unroll
            for (int k = 1; k < 4; ++k)
                v += *(const f32x4 *)&lds_o[k][r][d];
            if (whole) {
                if (d < hd) {
                    const int rr = t.row0 + r;
                    const int sees = t.shared ? t.len : per + over_group(b, rr);
                    const bool empty = sees <= 0 && !t.pre_len;
                    float out[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        out[k] = empty ? 0.f : v[k] / sum;
                    const int64_t token = row_token(b, t, rr);
                    put4((T *)a.y + (token * heads + head * b.group + (rr - over_group(b, rr) * b.group)) * hd + d, out, vec);
                }
            } else {
                *(f32x4 *)(a.parts[0] + (slot * kNarrowRows + r) * DP + d) = v;
                if (d == 0) {
                    a.sums[0][(slot * kNarrowRows + r) * 2] = top;
                    a.sums[0][(slot * kNarrowRows + r) * 2 + 1] = sum;
                }
            }
        }
        __syncthreads();
        at = base + u1;
    }
}

// Four results of a block from register r on, times f.
__device__ __forceinline__ f32x16 scaled(f32x16 v, int r, f32x4 f)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[r + i] *= f[i];
    return v;
}

// ---------------------------------------------------------------------------
// wide tiles: 128 rows, four waves on 32 rows each of a unit of 64 tokens
//
// For rows enough that the products are the work.  Blocks of 32 tokens stand in LDS in the order of
// the cache, as bf16, three of keys and three of values in turn: the waves read one while the next
// are on their way.  Operands are 32 lanes of 16 neighbouring bytes, free of bank conflicts.  Codes
// land in LDS as they are, two blocks further ahead, and the waves turn them into bf16 there, each
// code once for all 128 rows (through registers instead: 437 to 510 us against 312).
//
// Two workgroups a CU, so a SIMD has two waves: the scores of one block are formed beside the weights
// of the block before it, and one wave's exponentials beside the other's products.  Prompts of 64
// heads over 4096 shared and up to 1024 own tokens: 1210 us (970 TFLOP/s of what rows see; matrix
// cores busy 0.48 of the time, vector instructions issued 0.50, LDS reading 0.24: none is full); 16
// prefixes of 16,384 in int8 under 512 requests: 312 us (880 TFLOP/s).  Not kept: units of 64 tokens
// at once (spills, 1700 us and more), two chains of sums for the scores (+1%), operands six
// instructions ahead (none).  Weights are one bf16 here: in two parts, with a second product for what the
// first leaves, the prompts take 1765 us (1273 without), the int8 requests 618 (526), prompts at 64 dims 1055 (777),
// for an error of 0.0017 instead of 0.0024.
template <int KIND, int DP>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attend_wide_kernel(AttendArgs a)
{
    typedef uint16_t T;
    typedef Frag<T> F;
    constexpr int NS = DP / 16, ND = DP / 32;
    constexpr int kSide = kBlock * DP * 2;                   // bytes of a block's keys, and of its values
    constexpr bool CODED = KIND != kCacheNative;
    constexpr int kCodes = CODED ? kBlock * DP : kSide;      // of them as the cache holds them
    constexpr int kRaw = 6 * kSide, kScales = kRaw + (CODED ? 6 * kCodes : 0);
    // three blocks of keys, three of values; three of their codes, the scales of eight
    __shared__ alignas(16) char lds[kScales + (CODED ? 8 * 2 * kBlock * 4 : 0)];
    // direct loads of a wave for a block's keys and another's values
    constexpr int kLoads = (2 * kCodes / 1024 + 3) / 4 + (CODED ? 1 : 0);
    const AttendBatch &b = a.b;
    const int w = worker_of_block();
    const AttendList list = scalar(&b.plan->list[1]);
    const int first = scalar(b.start[1] + w);                // stale if the worker has no work
    const int64_t total = scalar(&b.plan->bad) ? 0 : (int64_t)list.units * b.kv_heads;
    int64_t at = (int64_t)w * list.run;
    const int64_t end = at + list.run < total ? at + list.run : total;
    if (at >= end)
        return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, h = lane >> 5, n = lane & 31;
    const int heads = b.group * b.kv_heads, hd = a.c.head_dim;
    const int in_page = (1 << (a.c.page_shift - 5)) - 1;
    const bool vec = (((uintptr_t)a.q | (uintptr_t)a.y) & 15) == 0;
    // row r of a result holds token 16 (r / 16) + 8 h + 0..7 in its registers when the rows of
    // the operand take the tokens with bits 2 and 3 of their number exchanged
    const int ktok = (n & 19) | (n & 4) << 1 | (n & 8) >> 1;
    int head = __builtin_amdgcn_readfirstlane(div_small(at, list.units)), x = first;

    for (; at < end; ++x) {
        if (x == list.tiles) {
            x = 0;
            ++head;
        }
        const AttendTile t = scalar(b.tiles[1] + x);
        const int64_t base = (int64_t)head * list.units + t.unit0;
        const int u0 = (int)(at - base);
        const int u1 = (int)((end < base + t.units ? end : base + t.units) - base);

        const int wr = wave * 32;                            // the wave's first row of the tile
        const bool works = wr < t.rows;
        const int wl = t.rows < wr + 32 ? t.rows - 1 : wr + 31;   // its last
        const bool mine = wr + n < t.rows;
        const int row = t.row0 + (mine ? wr + n : works ? wl : 0);
        F q[NS];
        {
            const int token = row_token(b, t, row);
            const T *p = (const T *)a.q + ((int64_t)token * heads + head * b.group + (row - over_group(b, row) * b.group)) * hd;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int d = 16 * s + 8 * h;
                q[s] = F{};
                if (mine && d < hd)
                    q[s] = q_frag<T>(p + d, vec);
            }
        }
        // own tokens that this lane's row sees, the most of the wave's rows, the fewest and the most of the tile's
        const int per = t.shared ? 0 : t.len - t.q_len + 1;
        const int see = t.shared ? t.len : per + over_group(b, row);
        const int see_wave = t.shared ? t.len : per + over_group(b, t.row0 + (works ? wl : 0));
        const int see_min = t.shared ? t.len : per + over_group(b, t.row0);
        const int see_max = t.shared ? t.len : per + over_group(b, t.row0 + t.rows - 1);
        // Blocks of 32 tokens, those of the prefix first: b0..b1-1 are the run's; every row sees whole
        // those before pre_full, and from pre_end on those before own_full.
        constexpr int kPer = kWideUnit / kBlock;
        const int b0 = u0 * kPer, b1 = u1 * kPer, pre_end = units_for(t.pre_len, kWideUnit) * kPer;
        const int pre_full = t.pre_len / kBlock, own_full = pre_end + (see_min > 0 ? see_min / kBlock : 0);
        const int32_t *own_pages = t.shared ? b.prefix_pages + (int64_t)t.seq * b.prefix_max_pages
                                            : b.pages + (int64_t)t.seq * b.max_pages;
        const int32_t *pre_pages = b.prefix_pages + (t.pre_len ? (int64_t)t.pre_seq * b.prefix_max_pages : 0);

        // Where blocks are: each lane holds the address of one, 64 at a time, so that the loop has no
        // address to form and no load to wait for.  Blocks past the run or that no row sees have the
        // cache's first page.
        bool lost = false;                                   // a page was not one of the cache's
        uint32_t far_lo = 0, far_hi = 0;
        int far0 = 0;
        auto look = [&](int k) __attribute__((always_inline)) {
            far0 = k;
            const int kk = k + lane;
            const bool in_pre = kk < pre_end;
            const int blk = in_pre ? kk : kk - pre_end, most = in_pre ? t.pre_len : see_max;
            int page = 0;
            if (kk < b1 && blk < units_for(most > 0 ? most : 0, kBlock))
                page = (in_pre ? pre_pages : own_pages)[blk >> (a.c.page_shift - 5)];
            const bool good = (uint32_t)page < (uint32_t)a.c.pages;
            lost |= __any(!good);
            const uint64_t p = (uint64_t)(a.c.base + cache_block(a.c, good ? page : 0, head, blk & in_page));
            far_lo = (uint32_t)p;
            far_hi = (uint32_t)(p >> 32);
        };
        auto block_of = [&](int k) __attribute__((always_inline)) -> const char * {
            if (k - far0 >= 64)
                look(k);
            const uint32_t lo = __builtin_amdgcn_readlane(far_lo, k - far0), hi = __builtin_amdgcn_readlane(far_hi, k - far0);
            return (const char *)((uint64_t)hi << 32 | lo);
        };
        // Places of the blocks k, k + 1 and k + 2 in LDS, three in turn; the fourth takes the first's.
        const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
        int at0 = 0, at1 = kSide, at2 = 2 * kSide;
        constexpr int kValues = 3 * kSide;                   // values behind the keys
        // Keys of block k with the values of the block before it, straight into LDS, as many loads from
        // every wave.  Codes go to a place of their own, three in turn too, with the scales of block k;
        // they become bf16 two blocks later.
        int raw0 = kRaw, raw1 = kRaw + 2 * kCodes, raw2 = kRaw + 4 * kCodes;
        auto fetch = [&](int k, const char *keys, const char *values, int key_to, int value_to) __attribute__((always_inline)) {
            constexpr int kPieces = kCodes / 1024;
            keys = scalar_address(keys);
            values = scalar_address(values);
#pragma unroll
            for (int i = 0; i < (2 * kPieces + 3) / 4; ++i) {
                // a wave without a piece of its own fetches another's again
                const int any = wave + 4 * i, piece = 2 * kPieces % 4 && any >= 2 * kPieces ? 2 * kPieces - 1 : any;
                const int side = kPieces % 4 ? piece >= kPieces : 4 * i >= kPieces, at = (piece - side * kPieces) * 1024;
                dma16_off(side ? values : keys, (uint32_t)(side * kCodes + at + lane * 16),
                          lds_at + (side ? value_to : key_to) + at);
            }
            if constexpr (CODED)
                dma4_off(keys, (uint32_t)(2 * kCodes + lane * 4), lds_at + kScales + (k & 7) * 2 * kBlock * 4);
        };
        // Codes at a place become keys and values in bf16, eight at a time: a thread's 8 bytes become
        // neighbouring 16 (16 and 32 would put every two lanes of a write on the same banks).
        constexpr int kEights = kBlock * DP / 8, NC = (kEights + 255) / 256;   // of a side; a thread's
        struct Codes { uint2 r[2][NC]; };
        auto pick = [&](int from) __attribute__((always_inline)) {
            Codes x;
            if constexpr (CODED)
#pragma unroll
                for (int side = 0; side < 2; ++side)
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        if (NC * 256 == kEights || tid + 256 * c < kEights)
                            x.r[side][c] = *(const uint2 *)(lds + from + side * kCodes + (tid + 256 * c) * 8);
            return x;
        };
        auto settle = [&](const Codes &x, int key_to, int value_to) __attribute__((always_inline)) {
            if constexpr (CODED)
#pragma unroll
                for (int side = 0; side < 2; ++side)
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        if (NC * 256 != kEights && tid + 256 * c >= kEights)
                            continue;
                        const Held<T, CODED ? KIND : kCacheInt8> eight{x.r[side][c]};
                        *(bf16x8 *)(lds + (side ? value_to : key_to) + (tid + 256 * c) * 16) = frag_of(eight).v;
                    }
        };

        f32x16 o[ND];
#pragma unroll
        for (int d = 0; d < ND; ++d)
            o[d] = f32x16{};
        float m = kNone, l = 0;
        // Raise the maximum to a lane's highest score if it is passed by far.
        auto raise = [&](const f32x16 &st) __attribute__((always_inline)) {
            float top = kNone;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                top = __builtin_fmaxf(top, st[r]);
            const auto halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
            top = __builtin_fmaxf(__uint_as_float(halves[0]), __uint_as_float(halves[1]));
            top *= a.scale;
            if (__any(top > m + kRaise)) {
                const float up = __builtin_fmaxf(m, top);
                const float f = up == kNone ? 1.f : fexp2(m - up);
                m = up;
                l *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    o[d] *= f;
            }
        };
        // Scores of a block, over the scale of q . k; of codes once rescaled.
        auto scores = [&](int at) __attribute__((always_inline)) {
            const char *kb = lds + at;
            f32x16 st{};
#pragma unroll
            for (int s = 0; s < NS; ++s)
                st = mma(F{*(const bf16x8 *)(kb + ((2 * s + h) * kBlock + ktok) * 16)}, q[s], st);
            return st;
        };
        auto rescale = [&](f32x16 &st, int side, int k) __attribute__((always_inline)) {
            if constexpr (CODED) {
                const float *sc = (const float *)(lds + kScales) + ((k & 7) * 2 + side) * kBlock;
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    st = scaled(st, r, *(const f32x4 *)&sc[16 * (r >> 3) + 8 * h + (r & 7)]);
            }
        };
        auto weights = [&](f32x16 &st) __attribute__((always_inline)) {
            const float off = m == kNone ? 0.f : -m;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                st[r] = fexp2(fmaf(st[r], a.scale, off));
                l += st[r];
            }
        };
        auto operand = [&](const f32x16 &st, int c) __attribute__((always_inline)) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = st[8 * c + i];
            return to_frag(v, T());
        };
        auto value = [&](int c, int d) __attribute__((always_inline)) {
            return F{*(const bf16x8 *)(lds + kValues + at0 + ((2 * c + h) * DP + 32 * d + n) * 16)};
        };
        auto add_values = [&](const f32x16 &st) __attribute__((always_inline)) {
            const F p[2] = {operand(st, 0), operand(st, 1)};
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    o[d] = mma(value(c, d), p[c], o[d]);
        };
        // Block k's weights and values with block k + 1's scores, laid out by hand: a fourth of the operands
        // ahead of the matrix instructions, and vector work behind each of those, which runs beside it.
        auto both = [&](f32x16 &cur, int k) __attribute__((always_inline)) {
            constexpr int kAhead = 4;
            const char *kb = lds + at1;
            const float off = m == kNone ? 0.f : -m;
            auto key = [&](int s) { return F{*(const bf16x8 *)(kb + ((2 * s + h) * kBlock + ktok) * 16)}; };
            F x[kAhead];
#pragma unroll
            for (int s = 0; s < kAhead; ++s)
                x[s] = key(s);
            f32x16 nxt{};
            F p[2];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                __builtin_amdgcn_sched_barrier(0);
                nxt = mma(x[s % kAhead], q[s], nxt);
                x[s % kAhead] = s + kAhead < NS ? key(s + kAhead)
                                                : value((s + kAhead - NS) / ND, (s + kAhead - NS) % ND);
#pragma unroll
                for (int r = 16 * s / NS; r < 16 * (s + 1) / NS; ++r) {
                    cur[r] = fexp2(fmaf(cur[r], a.scale, off));
                    l += cur[r];
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            rescale(cur, 1, k);
            rescale(nxt, 0, k + 1);
            p[0] = operand(cur, 0);
            p[1] = operand(cur, 1);
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                const int at = (NS + i) % kAhead;
                o[i % ND] = mma(x[at], p[i / ND], o[i % ND]);
                if (i + kAhead < NS)
                    x[at] = value((i + kAhead) / ND, (i + kAhead) % ND);
            }
            __builtin_amdgcn_sched_barrier(0);
            return nxt;
        };
        // A block of which some rows do not see all tokens.
        auto edge = [&](int k) __attribute__((always_inline)) {
            const bool in_pre = k < pre_end;
            const int tok0 = (in_pre ? k : k - pre_end) * kBlock;
            const int here = (in_pre ? t.pre_len : see) - tok0;          // tokens from the block on that this row sees
            const int most = (in_pre ? t.pre_len : see_wave) - tok0;     // that any row of the wave does
            if (most <= 0)
                return;
            f32x16 st = scores(at0);
            rescale(st, 0, k);
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (16 * (r >> 3) + 8 * h + (r & 7) >= here)
                    st[r] = kNone;
            raise(st);
            weights(st);
            rescale(st, 1, k);
            if constexpr (CODED)                             // a hidden token's scale may be NaN
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (16 * (r >> 3) + 8 * h + (r & 7) >= here)
                        st[r] = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int first = 16 * c + 8 * h;
                const F p = operand(st, c);
                F sees{};
                if constexpr (!CODED)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sees.v[i] = first + i < here ? 1.f : 0.f;
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    F v = value(c, d);
                    cut(v, most - first);                    // what no row sees may hold anything
                    if constexpr (!CODED)
                        odd_values<T>(v, sees, o[d]);
                    o[d] = mma(v, p, o[d]);
                }
            }
        };

        // At the start of block k its keys (if not used yet) and values and the next one's keys are there,
        // and one fetch is under way: keys are fetched three blocks ahead, values two.
        auto wait = [&]() __attribute__((always_inline)) {
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLoads) : "memory");
        };
        look(b0);
        const char *before = block_of(b0), *behind = before; // of the last two blocks fetched
        auto next = [&](int k) __attribute__((always_inline)) {
            before = behind;
            behind = block_of(k);
        };
        fetch(b0, behind, before, CODED ? raw0 : at0, CODED ? raw0 + kCodes : kValues + at2);   // the values are of no block
        next(b0 + 1);
        fetch(b0 + 1, behind, before, CODED ? raw1 : at1, CODED ? raw1 + kCodes : kValues + at0);
        next(b0 + 2);
        fetch(b0 + 2, behind, before, CODED ? raw2 : at2, CODED ? raw2 + kCodes : kValues + at1);
        if constexpr (CODED) {
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            settle(pick(raw0), at0, kValues + at2);
            settle(pick(raw1), at1, kValues + at0);
            settle(pick(raw2), at2, kValues + at1);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            next(b0 + 3);
            fetch(b0 + 3, behind, before, raw0, raw0 + kCodes);
            next(b0 + 4);
            fetch(b0 + 4, behind, before, raw1, raw1 + kCodes);
        }
        // Block k's place goes to block k + 3's keys, and codes two further.
        auto ahead = [&](int k) __attribute__((always_inline)) {
            next(k + (CODED ? 5 : 3));
            fetch(k + 5, behind, before, CODED ? raw2 : at0, CODED ? raw2 + kCodes : kValues + at2);
            return pick(raw0);
        };
        auto pass = [&](const Codes &x) __attribute__((always_inline)) {
            settle(x, at0, kValues + at2);
            int first = at0;
            at0 = at1;
            at1 = at2;
            at2 = first;
            first = raw0;
            raw0 = raw1;
            raw1 = raw2;
            raw2 = first;
        };
        for (int k = b0; k < b1;) {
            wait();
            const int full = k < pre_end ? pre_full : own_full;
            const int stop = full < b1 ? full : b1;
            if (k < stop) {
                f32x16 cur = scores(at0);
                rescale(cur, 0, k);
                raise(cur);
                for (; k + 1 < stop; ++k) {
                    wait();                                  // all waves are done with block k's keys
                    const Codes x = ahead(k);
                    __builtin_amdgcn_s_setprio(1);           // before the other workgroup's wave and its softmax
                    cur = both(cur, k);
                    __builtin_amdgcn_s_setprio(0);
                    raise(cur);
                    pass(x);
                }
                wait();
                const Codes x = ahead(k);
                weights(cur);
                rescale(cur, 1, k);
                add_values(cur);
                pass(x);
                ++k;
            } else {
                if (works)
                    edge(k);
                asm volatile("s_barrier" ::: "memory");      // its keys' place is free
                pass(ahead(k));
                ++k;
            }
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (lost) {
            l = __builtin_nanf("");
            if (!tid)
                atomicOr(b.flags, LORA_FLAG_CACHE_PAGE);
        }

        l += __shfl_xor(l, 32);
        const bool whole = t.kept < 0 && u0 == 0 && u1 == t.units;
        if (mine) {
            if (whole) {
                const bool empty = see <= 0 && !t.pre_len;
                const float by = empty ? 0.f : 1.f / l;
                const int64_t token = row_token(b, t, row);
                T *y = (T *)a.y + (token * heads + head * b.group + (row - over_group(b, row) * b.group)) * hd;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        const int dim = 32 * d + 2 * r + 4 * h;
                        float out[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            out[i] = empty ? 0.f : o[d][r + i] * by;
                        if (dim < hd)
                            put4(y + dim, out, vec);
                    }
            } else {
                const int64_t slot = part_slot(list, b.workers[1], head, t, w) * kWideRows + wr + n;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; r += 4)
                        *(f32x4 *)(a.parts[1] + slot * DP + 32 * d + 2 * r + 4 * h) =
                            f32x4{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]};
                if (!h) {
                    a.sums[1][slot * 2] = m;
                    a.sums[1][slot * 2 + 1] = l;
                }
            }
        }
        at = base + u1;
    }
}

// ---------------------------------------------------------------------------
// joining parts

// A workgroup takes a narrow tile of a key-value head, or 32 rows of a wide one, four dims a lane
// (starting workgroups counts: 16 long prompts take 34 us of joining, 39 with 16 rows each, and more with 8).
// A group of lanes takes a row, or a share of its parts where rows are few: each lane fetches the
// maximum and sum of one part, the weights follow from them, and no load of a part waits for
// another.  Wide tiles whose parts are kept only where workers part are found by those borders,
// which are far fewer than the tiles.  The chain tile, borders, maxima, values bounds it: 6 to 11 us
// where a worker's border parts a tile here and there, 30 us for 512 requests with prefixes and 34 us
// for 16 long prompts, which have some 67 MB of parts to read each.
// Where there are many narrow tiles of few rows, a workgroup takes several key-value heads of one.
struct JoinGrid {
    int32_t narrow, kept, borders;       // workgroups: narrow tiles, wide ones whose parts are kept, borders
    int32_t heads, each;                 // of a narrow tile: workgroups, and key-value heads a workgroup
};
constexpr int kJoinRows = 32, kJoinChunks = kWideRows / kJoinRows;

template <typename T, int DP>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, JoinGrid grid)
{
    constexpr int NL = DP <= 64 ? 16 : DP <= 128 ? 32 : 64, NG = 256 / NL;
    __shared__ f32x4 lds_o[NG][NL];
    __shared__ float lds_m[NG], lds_l[NG];
    __shared__ SimplePlan own;
    const AttendBatch &b = a.b;
    const int block = blockIdx.y * gridDim.x + blockIdx.x;   // rows of a grid: one holds 2^32 threads at most
    if (block >= grid.narrow + grid.kept + grid.borders)
        return;
    const int l = block >= grid.narrow;
    AttendList list, other{};
    AttendTile t;
    int head, chunk = 0, w0, w1;
    if (b.simple) {
        list = plan_simple(b, own);
        const int x = block / grid.heads;
        head = block % grid.heads;
        if (x >= list.tiles)
            return;
        t = simple_tile(x, own.len[x], b.group, own.unit0[x]);
    } else if (!l) {
        list = b.plan->list[0];
        other = b.plan->list[1];
        const int x = block / grid.heads;
        head = block % grid.heads;
        t = b.tiles[0][x];                                   // stale where x is past the list
        if (x >= list.tiles)
            return;
    } else {
        list = b.plan->list[1];
        other = b.plan->list[0];
        const int i = block - grid.narrow, kept = i < grid.kept;
        chunk = (kept ? i : i - grid.kept) % kJoinChunks;
        const int k = (kept ? i : i - grid.kept) / kJoinChunks;
        if (kept) {
            const int x = k / b.kv_heads;
            head = k % b.kv_heads;
            t = b.tiles[1][x];
            if (x >= list.tiles || t.kept < 0)
                return;
        } else {                                             // the first border inside of a tile
            const int64_t at = (int64_t)(k + 1) * list.run;
            if (at >= (int64_t)list.units * b.kv_heads)
                return;
            head = div_small(at, list.units);
            t = b.tiles[1][b.start[1][k + 1]];
            if (t.kept >= 0 || first_worker(list, head, t) != k)
                return;
        }
        if (chunk * kJoinRows >= t.rows)
            return;
    }
    if (t.shared)
        return;
    const int each = l ? 1 : grid.each, per_head = NG / each;            // heads, and groups of one
    const int grp = threadIdx.x / NL % per_head;
    head = head * each + threadIdx.x / NL / per_head;
    const bool has = head < b.kv_heads;
    w0 = has ? first_worker(list, head, t) : 0;
    w1 = has ? last_worker(list, head, t) : 0;
    const bool joins = has && (t.kept >= 0 || w0 != w1);
    if (each == 1 && !joins)
        return;
    const int R = list_rows(l), hd = a.c.head_dim, heads = b.group * b.kv_heads;
    PrefixTile pre{0, 0};
    int pre_row = 0;
    if (t.prefix >= 0) {
        pre = b.prefix_tile[t.prefix];
        const int lo = clamp_to(b.prefix_seqs[t.prefix], 0, b.n_seqs);
        pre_row = t.pre_row - b.list_before[lo] * b.group;
    }
    const AttendList shared = pre.list == l ? list : other;
    const int PR = list_rows(pre.list);
    const bool vec = ((uintptr_t)a.y & 15) == 0;
    int split = 1;                                           // groups of a row
    const int row_end = l && t.rows > (chunk + 1) * kJoinRows ? (chunk + 1) * kJoinRows : t.rows;
    const int row0 = chunk * kJoinRows;
    while (split < 8 && (row_end - row0) * split * 2 <= per_head)
        split *= 2;
    const int lane = threadIdx.x % NL, sub = grp % split, d = lane * 4;
    const int n_own = w1 - w0 + 1;
    const int64_t own_at = part_slot(list, b.workers[l], head, t, w0);
    for (int r0 = row0; r0 < row_end; r0 += per_head / split) {
        const int r = r0 + grp / split;
        const bool live = joins && r < row_end;
        float top = kNone, sum = 0;
        f32x4 v = {0, 0, 0, 0};
        if (live) {
            // the parts of the row: its own ones, then those over its prefix
            int n = n_own, pr = 0;
            int64_t pre_at = 0;
            if (t.prefix >= 0) {
                pr = pre_row + r;
                const AttendTile s = b.tiles[pre.list][pre.tile + pr / PR];
                const int s0 = first_worker(shared, head, s);
                n += last_worker(shared, head, s) - s0 + 1;
                pre_at = part_slot(shared, b.workers[pre.list], head, s, s0);
                pr %= PR;
            }
            for (int k0 = 0; k0 < n; k0 += NL * split) {
                const bool there = k0 + lane * split + sub < n;
                const int k = there ? k0 + lane * split + sub : 0;
                const bool mine = k < n_own;
                // of a tile that is not kept: its first worker's last part, the others' first
                const int64_t slot = mine ? (t.kept >= 0 ? own_at + k : k ? 2ll * (w0 + k) : own_at) : pre_at + (k - n_own);
                const int64_t at = mine ? slot * R + r : slot * PR + pr;
                float m = kNone, one = 0;
                if (there) {
                    const float2 ms = *(const float2 *)((mine ? a.sums[l] : a.sums[pre.list]) + at * 2);
                    m = ms.x;
                    one = ms.y;
                }
                float up = m;
#pragma unroll
                for (int i = 1; i < NL; i <<= 1)
                    up = __builtin_fmaxf(up, __shfl_xor(up, i, NL));
                up = __builtin_fmaxf(up, top);
                const float f = !there ? 0.f : m == kNone ? 1.f : fexp2(m - up), was = top == kNone ? 1.f : fexp2(top - up);
                one *= f;
#pragma unroll
                for (int i = 1; i < NL; i <<= 1)
                    one += __shfl_xor(one, i, NL);
                sum = sum * was + one;
                v *= was;
                top = up;
                const uint64_t from = (uint64_t)((mine ? a.parts[l] : a.parts[pre.list]) + at * DP);
                const int here = (n - k0 - sub + split - 1) / split, count = here < NL ? here : NL;
                for (int i0 = 0; i0 < count; i0 += 4)        // past the last: the row's first part, left out
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t lo = __shfl((uint32_t)from, i0 + i, NL), hi = __shfl((uint32_t)(from >> 32), i0 + i, NL);
                        const float by = __shfl(f, i0 + i, NL);
                        if (DP == 4 * NL || d < DP) {
                            const f32x4 o = *(const f32x4 *)(((uint64_t)hi << 32 | lo) + d * 4) * by;
                            v += i0 + i < count ? o : f32x4{0, 0, 0, 0};
                        }
                    }
            }
        }
        if (split > 1) {
            const int me = threadIdx.x / NL;
            lds_o[me][lane] = v;
            if (!lane) {
                lds_m[me] = top;
                lds_l[me] = sum;
            }
            __syncthreads();
            if (live && !sub) {
                float up = top;
                for (int k = 1; k < split; ++k)
                    up = __builtin_fmaxf(up, lds_m[me + k]);
                float f = top == kNone ? 1.f : fexp2(top - up);
                v *= f;
                sum *= f;
                for (int k = 1; k < split; ++k) {
                    f = lds_m[me + k] == kNone ? 1.f : fexp2(lds_m[me + k] - up);
                    v += lds_o[me + k][lane] * f;
                    sum += lds_l[me + k] * f;
                }
            }
        }
        if (live && !sub && d < hd) {
            const int rr = t.row0 + r;
            const bool empty = t.len - t.q_len + 1 + over_group(b, rr) <= 0 && !t.pre_len && t.prefix < 0;
            float out[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                out[k] = empty ? 0.f : v[k] / sum;
            put4((T *)a.y + ((int64_t)(t.token0 + over_group(b, rr)) * heads + head * b.group + (rr - over_group(b, rr) * b.group)) * hd + d,
                 out, vec);
        }
    }
}

template <typename T, int KIND>
hipError_t launch_narrow(const AttendArgs &a, hipStream_t st)
{
    switch (a.c.dp) {
    case 64: attend_narrow_kernel<T, KIND, 64><<<a.b.workers[0], 256, 0, st>>>(a); break;
    case 96: attend_narrow_kernel<T, KIND, 96><<<a.b.workers[0], 256, 0, st>>>(a); break;
    case 128: attend_narrow_kernel<T, KIND, 128><<<a.b.workers[0], 256, 0, st>>>(a); break;
    default: attend_narrow_kernel<T, KIND, 256><<<a.b.workers[0], 256, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

template <int KIND>
hipError_t launch_wide(const AttendArgs &a, hipStream_t st)
{
    switch (a.c.dp) {
    case 64: attend_wide_kernel<KIND, 64><<<a.b.workers[1], 256, 0, st>>>(a); break;
    case 96: attend_wide_kernel<KIND, 96><<<a.b.workers[1], 256, 0, st>>>(a); break;
    case 128: attend_wide_kernel<KIND, 128><<<a.b.workers[1], 256, 0, st>>>(a); break;
    default: attend_wide_kernel<KIND, 256><<<a.b.workers[1], 256, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_all(const AttendArgs &a, hipStream_t st)
{
    hipError_t e = hipSuccess;
    if (a.b.cap[1] && !a.b.simple)                           // of a simple batch nobody writes a list of wide tiles
        e = a.c.kind == kCacheNative ? launch_wide<kCacheNative>(a, st)
          : a.c.kind == kCacheFp8 ? launch_wide<kCacheFp8>(a, st)
                                  : launch_wide<kCacheInt8>(a, st);
    if (e != hipSuccess)
        return e;
    e = a.c.kind == kCacheNative ? launch_narrow<T, kCacheNative>(a, st)
                 : a.c.kind == kCacheFp8 ? launch_narrow<T, kCacheFp8>(a, st)
                                         : launch_narrow<T, kCacheInt8>(a, st);
    if (e != hipSuccess)
        return e;
    JoinGrid grid;
    // a workgroup has 1024 / dp groups of lanes (4, 8 or 16), a row each; a tile of one row for one head
    // costs as much as one that fills them
    const int groups = a.c.dp <= 64 ? 16 : a.c.dp <= 128 ? 8 : 4, rows = std::min(a.b.max_queries * a.b.group, kNarrowRows);
    grid.each = 1;
    while (a.b.cap[0] * a.b.kv_heads > 1024 * grid.each && grid.each * 2 <= a.b.kv_heads && grid.each * 2 * rows <= groups)
        grid.each *= 2;
    grid.heads = (a.b.kv_heads + grid.each - 1) / grid.each;
    grid.narrow = a.b.cap[0] * grid.heads;
    grid.kept = a.b.n_prefixes && a.b.group > kShareRows ? a.b.cap[1] * a.b.kv_heads * kJoinChunks : 0;
    grid.borders = a.b.cap[1] ? (a.b.workers[1] - 1) * kJoinChunks : 0;
    const int blocks = grid.narrow + grid.kept + grid.borders, across = std::min(blocks, 1 << 22);
    const dim3 all(across, (blocks + across - 1) / across);
    switch (a.c.dp) {
    case 64: attend_join_kernel<T, 64><<<all, 256, 0, st>>>(a, grid); break;
    case 96: attend_join_kernel<T, 96><<<all, 256, 0, st>>>(a, grid); break;
    case 128: attend_join_kernel<T, 128><<<all, 256, 0, st>>>(a, grid); break;
    default: attend_join_kernel<T, 256><<<all, 256, 0, st>>>(a, grid); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attend_plan(const AttendBatch &b, hipStream_t st)
{
    attend_plan_kernel<<<1, kPlanThreads, 0, st>>>(b);
    return hipGetLastError();
}

hipError_t launch_attend(bool bf16, const AttendArgs &a, hipStream_t st)
{
    return bf16 ? launch_all<uint16_t>(a, st) : launch_all<float>(a, st);
}

}  // namespace lora
