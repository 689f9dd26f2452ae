// lora_cache.hip -- gfx950 kernels that write keys and values into the paged cache and read
// them back.
//
// In 8 bits a head of a token has the scale max|x| / top (top 448 for fp8, 127 for int8) and the
// codes round(x top / max|x|), to the nearest, ties to even.  The quotient is exact before that
// rounding where it matters: for bf16 data it is rounded once to fp32 (a product with the
// reciprocal and one correction by the remainder, which fp32 holds), and a quotient of two 8-bit
// significands that is not a tie differs from one by far more than 2^-24; for fp32 data it is
// formed in double.
#include <hip/hip_runtime.h>

#include "lora_attend.h"

namespace lora {
namespace {

template <typename T, int N> struct alignas(sizeof(T) * N) Pack { T v[N]; };
typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;

__device__ __forceinline__ float value_of(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ void put_value(uint16_t &to, float f)
{
    __bf16 h = (__bf16)f;
    to = __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ void put_value(float &to, float f) { to = f; }

// How one head of a token is coded.
struct Coding {
    float scale;                 // a code's unit, NaN for a head with an infinity or NaN
    float high;                  // max|x|, at least 2^-100 (whose reciprocal fp32 still holds)
    float mant, inv, per;        // high shift in [1, 2), its reciprocal, top times that
    float shift;                 // a power of two
    bool odd;
};

template <int KIND>
__device__ __forceinline__ Coding coding_of(uint32_t high_bits)
{
    constexpr float top = KIND == kCacheFp8 ? 448.f : 127.f;
    Coding c;
    c.odd = high_bits >= 0x7f800000u;
    const float high = c.odd ? 1.f : __uint_as_float(high_bits);
    c.high = __builtin_fmaxf(high, 0x1p-100f);
    c.shift = ldexpf(1.f, 127 - (int)(__float_as_uint(c.high) >> 23));
    c.mant = c.high * c.shift;
    c.inv = 1.f / c.mant;
    c.per = top / c.mant;
    c.scale = c.odd ? __builtin_nanf("") : c.high / top;
    return c;
}

// x top / high rounded once to fp32, of bf16 values
template <int KIND>
__device__ __forceinline__ float level_of(const Coding &c, uint16_t raw)
{
    constexpr float top = KIND == kCacheFp8 ? 448.f : 127.f;
    const float x = value_of(raw) * c.shift;
    const float q = x * c.per;
    return fmaf(fmaf(-q, c.mant, x * top), c.inv, q);
}
// the same of fp32 values, rounded to fp32 so that a later rounding to fewer bits is that of the
// quotient itself: cut off, with the last bit set if anything was
template <int KIND>
__device__ __forceinline__ float level_of(const Coding &c, float x)
{
    constexpr double top = KIND == kCacheFp8 ? 448.0 : 127.0;
    const double q = (double)x * top / (double)c.high;
    float f = (float)q;
    uint32_t bits = __float_as_uint(f);
    if ((double)f != q) {
        if (fabs((double)f) > fabs(q))
            bits -= 1;
        bits |= 1;
    }
    return __uint_as_float(bits);
}

// Eight codes, as the bytes of two words.
template <int KIND>
__device__ __forceinline__ uint2 codes_of(const float *q)
{
    uint32_t r[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if constexpr (KIND == kCacheFp8) {
            int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * w], q[4 * w + 1], 0, false);
            r[w] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * w + 2], q[4 * w + 3], v, true);
        } else {
            // the sum is rounded to whole numbers, whose low byte its low bits hold
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = __float_as_uint(q[4 * w + i] + 12582912.f);
            r[w] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(v[3], v[2], 0x0c0c0400),
                                         __builtin_amdgcn_perm(v[1], v[0], 0x0c0c0400), 0x05040100);
        }
    }
    return make_uint2(r[0], r[1]);
}
template <int KIND>
__device__ __forceinline__ float code_value(uint8_t c)
{
    if constexpr (KIND == kCacheFp8)
        return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
    else
        return (float)(int8_t)c;
}

template <typename T>
__device__ __forceinline__ Pack<T, 8> load8(const T *p, bool vec)
{
    if (vec)
        return *(const Pack<T, 8> *)p;
    Pack<T, 8> r;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        r.v[j] = p[j];
    return r;
}

// A workgroup has a window of 32 tokens of the batch and one head, of its keys or of its values; 8
// lanes a token, a lane every eighth unit of 8 dims.  Keys move in units as they are.  Values stand
// in units of 8 tokens: where 8 tokens of the batch fill such a unit (an octet: consecutive slots
// from a multiple of 8 on) they pass through LDS and move as units, whatever their place in the
// batch; other tokens move an element at a time.  An octet is stored by the window with its first
// token, which fetches up to 7 tokens behind itself for it, and loaded by every window that it
// touches.  Prompts go at the rate of memory; single tokens of many requests write every 8th element of a
// run, 8 dims of bf16 or 16 codes to a line of 128 bytes.
//
// Store and load: 13,044 tokens of 32 heads of 128, bf16, 92 and 106 us (4.4 TB/s over both); 32,971
// of 8 heads, int8, 55 and 44 us (4.2 TB/s); with values moved an element at a time the two cases took
// 303 and 139 us.  512 single tokens of 8 heads, fp8, 8.2 and 5.4 us: the chain slots, data, maximum,
// codes, store, and the stores of single elements.
constexpr int kWindow = 32, kAround = 7;

// Workgroups equal mod 8 share an XCD: each XCD takes a run of neighbouring windows, which write
// parts of the same lines.
__device__ __forceinline__ int window_of_block() { return (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3); }

struct Window {
    int32_t slot[kWindow + 2 * kAround];     // from 7 tokens before the window on; -1: none
};

// The slots around a window; those past the cache count as none and are flagged.
__device__ __forceinline__ void fill_window(const CacheArgs &a, Window &w, int window)
{
    if (threadIdx.x < kWindow + 2 * kAround) {
        const int t = window * kWindow - kAround + (int)threadIdx.x;
        int s = t >= 0 && t < a.T ? a.slots[t] : -1;
        if (s >= 0 && (s >> a.c.page_shift) >= a.c.pages) {
            if (threadIdx.x >= kAround && threadIdx.x < kAround + kWindow)
                atomicOr(a.flags, LORA_FLAG_CACHE_SLOT);
            s = -1;
        }
        w.slot[threadIdx.x] = s < 0 ? -1 : s;
    }
    __syncthreads();
}
// Whether the octet from place p on (p + 7 inside of the array) is whole.
__device__ __forceinline__ bool octet_at(const Window &w, int p)
{
    const int s = w.slot[p];
    bool all = s >= 0 && !(s & 7);
#pragma unroll
    for (int j = 1; j < 8; ++j)
        all &= w.slot[p + j] == s + j;
    return all;
}
__device__ __forceinline__ char *block_at(const CacheArgs &a, int slot, int head)
{
    const int in_page = slot & ((1 << a.c.page_shift) - 1);
    return a.c.base + cache_block(a.c, slot >> a.c.page_shift, head, in_page >> 5);
}

// Eight words, of one token each, against as many units of 8 elements of one dim each.
template <int ELEM>
__device__ __forceinline__ void turn(const uint32_t (&w)[8], uint32_t (&u)[8])
{
    if constexpr (ELEM == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            u[j] = w[j];
    } else if constexpr (ELEM == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], 0x05040100);
            u[4 + j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], 0x07060302);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t lo0 = __builtin_amdgcn_perm(w[4 * j + 1], w[4 * j], 0x05010400);
            const uint32_t hi0 = __builtin_amdgcn_perm(w[4 * j + 1], w[4 * j], 0x07030602);
            const uint32_t lo1 = __builtin_amdgcn_perm(w[4 * j + 3], w[4 * j + 2], 0x05010400);
            const uint32_t hi1 = __builtin_amdgcn_perm(w[4 * j + 3], w[4 * j + 2], 0x07030602);
            u[j] = __builtin_amdgcn_perm(lo1, lo0, 0x05040100);
            u[2 + j] = __builtin_amdgcn_perm(lo1, lo0, 0x07060302);
            u[4 + j] = __builtin_amdgcn_perm(hi1, hi0, 0x05040100);
            u[6 + j] = __builtin_amdgcn_perm(hi1, hi0, 0x07060302);
        }
    }
}
// And back.
template <int ELEM>
__device__ __forceinline__ void turn_back(const uint32_t (&u)[8], uint32_t (&w)[8])
{
    if constexpr (ELEM == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = u[j];
    } else if constexpr (ELEM == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[2 * j] = __builtin_amdgcn_perm(u[4 + j], u[j], 0x05040100);
            w[2 * j + 1] = __builtin_amdgcn_perm(u[4 + j], u[j], 0x07060302);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t lo0 = __builtin_amdgcn_perm(u[2 + j], u[j], 0x05010400);
            const uint32_t hi0 = __builtin_amdgcn_perm(u[2 + j], u[j], 0x07030602);
            const uint32_t lo1 = __builtin_amdgcn_perm(u[6 + j], u[4 + j], 0x05010400);
            const uint32_t hi1 = __builtin_amdgcn_perm(u[6 + j], u[4 + j], 0x07030602);
            w[4 * j] = __builtin_amdgcn_perm(lo1, lo0, 0x05040100);
            w[4 * j + 1] = __builtin_amdgcn_perm(lo1, lo0, 0x07060302);
            w[4 * j + 2] = __builtin_amdgcn_perm(hi1, hi0, 0x05040100);
            w[4 * j + 3] = __builtin_amdgcn_perm(hi1, hi0, 0x07060302);
        }
    }
}

// One token's head as the cache holds it, in units.
template <typename T, int KIND> struct HeldUnit;
template <> struct HeldUnit<uint16_t, kCacheNative> { typedef Pack<uint16_t, 8> type; typedef uint16_t elem; };
template <> struct HeldUnit<float, kCacheNative> { typedef Pack<float, 8> type; typedef float elem; };
template <typename T> struct HeldUnit<T, kCacheFp8> { typedef Pack<uint8_t, 8> type; typedef uint8_t elem; };
template <typename T> struct HeldUnit<T, kCacheInt8> { typedef Pack<uint8_t, 8> type; typedef uint8_t elem; };

// The 8 lanes of a token read its head.
template <typename T, int NU>
__device__ __forceinline__ void read_head(const T *x, int units, int part, bool vec, Pack<T, 8> (&p)[NU])
{
#pragma unroll
    for (int n = 0; n < NU; ++n)
        if (part + 8 * n < units)
            p[n] = load8(x + 8 * (part + 8 * n), vec);
}

// They code it; *scale is what the codes are in.
template <typename T, int KIND, int NU>
__device__ __forceinline__ void code_head(const Pack<T, 8> (&p)[NU], int units, int part,
                                          typename HeldUnit<T, KIND>::type (&out)[NU], float *scale)
{
    if constexpr (KIND == kCacheNative) {
#pragma unroll
        for (int n = 0; n < NU; ++n)
            out[n] = p[n];
    } else {
        // the largest of the bits without sign is the largest size, NaN above infinity
        uint32_t high = 0;
        if constexpr (sizeof(T) == 2) {
            u16x2 top = {0, 0};
#pragma unroll
            for (int n = 0; n < NU; ++n)
                if (part + 8 * n < units)
#pragma unroll
                    for (int j = 0; j < 8; j += 2)
                        top = __builtin_elementwise_max(top, u16x2{p[n].v[j], p[n].v[j + 1]} & u16x2{0x7fff, 0x7fff});
            high = (uint32_t)(top[0] > top[1] ? top[0] : top[1]) << 16;
        } else {
#pragma unroll
            for (int n = 0; n < NU; ++n)
                if (part + 8 * n < units)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t bits = __float_as_uint(p[n].v[j]) & 0x7fffffffu;
                        high = bits > high ? bits : high;
                    }
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
            const uint32_t o = __shfl_xor(high, d);
            high = o > high ? o : high;
        }
        const Coding c = coding_of<KIND>(high);
        *scale = c.scale;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[j] = c.odd || part + 8 * n >= units ? 0.f : level_of<KIND>(c, p[n].v[j]);
            out[n] = __builtin_bit_cast(typename HeldUnit<T, KIND>::type, codes_of<KIND>(q));
        }
    }
}

template <typename T, int KIND, int NU>
__global__ __launch_bounds__(256) void cache_store_kernel(CacheArgs a)
{
    typedef typename HeldUnit<T, KIND>::type U;
    typedef typename HeldUnit<T, KIND>::elem E;
    constexpr int kRow = NU * 64 * (int)sizeof(E) + 16;              // of a token in LDS
    __shared__ Window win;
    __shared__ alignas(16) char rows[kWindow + kAround][kRow];
    const int window = window_of_block();
    if (window * kWindow >= a.T)
        return;
    const int i = threadIdx.x >> 3, part = threadIdx.x & 7, head = blockIdx.y, side = blockIdx.z;
    const int hd = a.c.head_dim, units = hd >> 3;
    const T *x = (const T *)(side ? a.v_in : a.k_in) + head * hd;
    const int64_t stride = (int64_t)a.c.kv_heads * hd, t0 = (int64_t)window * kWindow;
    const bool vec = ((uintptr_t)(side ? a.v_in : a.k_in) & 15) == 0;
    Pack<T, 8> p[NU];                        // on their way while the slots are
    if (t0 + i < a.T)
        read_head<T, NU>(x + (t0 + i) * stride, units, part, vec, p);
    fill_window(a, win, window);
    const int s = win.slot[kAround + i], tok = s & (kBlock - 1);
    U u[NU];
    float scale = 0;
    if (s >= 0) {
        char *blk = block_at(a, s, head);
        code_head<T, KIND, NU>(p, units, part, u, &scale);
        if (KIND != kCacheNative && !part)
            ((float *)(blk + 2 * a.c.half))[side * kBlock + tok] = scale;
        const bool octet = side && octet_at(win, kAround + i - (s & 7));
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int at = part + 8 * n;
            if (at >= units)
                continue;
            if (!side) {
                *(U *)((E *)blk + key_at(tok, 8 * at)) = u[n];
            } else if (octet) {
                *(U *)(rows[i] + at * sizeof(U)) = u[n];
            } else {
                E *y = (E *)(blk + a.c.half);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[value_at(a.c.dp, tok, 8 * at + j)] = u[n].v[j];
            }
        }
    }
    if (!side)
        return;
    // tokens behind the window of octets that start in it
    if (i < kAround) {
        const int s2 = win.slot[kAround + kWindow + i], r = s2 & 7;
        if (s2 >= 0 && r > i && octet_at(win, kAround + kWindow + i - r)) {
            read_head<T, NU>(x + (t0 + kWindow + i) * stride, units, part, vec, p);
            code_head<T, KIND, NU>(p, units, part, u, &scale);
#pragma unroll
            for (int n = 0; n < NU; ++n)
                if (part + 8 * n < units)
                    *(U *)(rows[kWindow + i] + (part + 8 * n) * sizeof(U)) = u[n];
        }
    }
    const int lane = threadIdx.x & 63;
    uint64_t starts = __ballot(lane < kWindow && octet_at(win, kAround + (lane & 31)));
    __syncthreads();
    const int words = hd * (int)sizeof(E) / 4;
    for (int k = threadIdx.x; starts; k += 256) {
        while (starts && k >= words) {
            k -= words;
            starts &= starts - 1;
        }
        if (!starts)
            break;
        const int first = __builtin_ctzll(starts), slot = win.slot[kAround + first];
        uint32_t w[8], o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = *(const uint32_t *)(rows[first + j] + 4 * k);
        turn<sizeof(E)>(w, o);
        char *y = block_at(a, slot, head) + a.c.half +
                  value_at(a.c.dp, slot & (kBlock - 1), k * (4 / (int)sizeof(E))) * (int)sizeof(E);
        *(uint4 *)y = make_uint4(o[0], o[1], o[2], o[3]);
        *(uint4 *)(y + 16) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

template <typename T, int KIND, int NU>
__global__ __launch_bounds__(256) void cache_load_kernel(CacheArgs a)
{
    typedef typename HeldUnit<T, KIND>::type U;
    typedef typename HeldUnit<T, KIND>::elem E;
    constexpr int kRow = NU * 64 * (int)sizeof(E) + 16;
    __shared__ Window win;
    __shared__ alignas(16) char rows[kWindow][kRow];
    const int window = window_of_block();
    if (window * kWindow >= a.T)
        return;
    const int i = threadIdx.x >> 3, part = threadIdx.x & 7, head = blockIdx.y, side = blockIdx.z;
    const int hd = a.c.head_dim, units = hd >> 3;
    fill_window(a, win, window);
    if (side) {
        const int lane = threadIdx.x & 63;
        uint64_t starts = __ballot(lane < kWindow + kAround && octet_at(win, lane < kWindow + kAround ? lane : 0));
        const int words = hd * (int)sizeof(E) / 4;
        for (int k = threadIdx.x; starts; k += 256) {
            while (starts && k >= words) {
                k -= words;
                starts &= starts - 1;
            }
            if (!starts)
                break;
            const int first = __builtin_ctzll(starts), slot = win.slot[first];
            const char *x = block_at(a, slot, head) + a.c.half +
                            value_at(a.c.dp, slot & (kBlock - 1), k * (4 / (int)sizeof(E))) * (int)sizeof(E);
            const uint4 lo = *(const uint4 *)x, hi = *(const uint4 *)(x + 16);
            const uint32_t o[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t w[8];
            turn_back<sizeof(E)>(o, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int to = first + j - kAround;
                if (to >= 0 && to < kWindow)
                    *(uint32_t *)(rows[to] + 4 * k) = w[j];
            }
        }
        __syncthreads();
    }
    const int s = win.slot[kAround + i], tok = s & (kBlock - 1);
    if (s < 0)
        return;
    const char *blk = block_at(a, s, head);
    const bool octet = side && octet_at(win, kAround + i - (s & 7));
    T *y = (T *)(side ? a.v_out : a.k_out) + ((int64_t)((int64_t)window * kWindow + i) * a.c.kv_heads + head) * hd;
    const bool vec = ((uintptr_t)(side ? a.v_out : a.k_out) & 15) == 0;
    float scale = 1.f;
    if constexpr (KIND != kCacheNative)
        scale = ((const float *)(blk + 2 * a.c.half))[side * kBlock + tok];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        const int at = part + 8 * n;
        if (at >= units)
            continue;
        U u;
        if (!side) {
            u = *(const U *)((const E *)blk + key_at(tok, 8 * at));
        } else if (octet) {
            u = *(const U *)(rows[i] + at * sizeof(U));
        } else {
            const E *x = (const E *)(blk + a.c.half);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                u.v[j] = x[value_at(a.c.dp, tok, 8 * at + j)];
        }
        Pack<T, 8> p;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (KIND == kCacheNative)
                p.v[j] = u.v[j];
            else
                put_value(p.v[j], scale * code_value<KIND>(u.v[j]));
        }
        if (vec) {
            *(Pack<T, 8> *)(y + 8 * at) = p;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[8 * at + j] = p.v[j];
        }
    }
}

template <typename T, int KIND, int NU>
hipError_t launch(bool store, const CacheArgs &a, hipStream_t st)
{
    const dim3 grid(((a.T + kWindow - 1) / kWindow + 7) / 8 * 8, a.c.kv_heads, 2);
    if (store)
        cache_store_kernel<T, KIND, NU><<<grid, 256, 0, st>>>(a);
    else
        cache_load_kernel<T, KIND, NU><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
}

template <typename T, int KIND>
hipError_t launch_units(bool store, const CacheArgs &a, hipStream_t st)
{
    if (a.c.head_dim <= 64)
        return launch<T, KIND, 1>(store, a, st);
    if (a.c.head_dim <= 128)
        return launch<T, KIND, 2>(store, a, st);
    return launch<T, KIND, 4>(store, a, st);
}

template <typename T>
hipError_t launch_kind(bool store, const CacheArgs &a, hipStream_t st)
{
    return a.c.kind == kCacheNative ? launch_units<T, kCacheNative>(store, a, st)
         : a.c.kind == kCacheFp8 ? launch_units<T, kCacheFp8>(store, a, st)
                                 : launch_units<T, kCacheInt8>(store, a, st);
}

}  // namespace

hipError_t launch_cache_store(bool bf16, const CacheArgs &a, hipStream_t st)
{
    return bf16 ? launch_kind<uint16_t>(true, a, st) : launch_kind<float>(true, a, st);
}

hipError_t launch_cache_load(bool bf16, const CacheArgs &a, hipStream_t st)
{
    return bf16 ? launch_kind<uint16_t>(false, a, st) : launch_kind<float>(false, a, st);
}

}  // namespace lora
