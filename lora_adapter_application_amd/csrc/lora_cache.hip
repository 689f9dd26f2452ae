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

__device__ __forceinline__ float value_of(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float value_of(float v) { return v; }
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
    float mant, inv, per;        // high / 2^exp in [1, 2), its reciprocal, top times that
    int exp;
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
    c.exp = (int)(__float_as_uint(c.high) >> 23) - 127;
    c.mant = ldexpf(c.high, -c.exp);
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
    const float x = ldexpf(value_of(raw), -c.exp);
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
            r[w] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r[w] |= ((uint32_t)(int)rintf(q[4 * w + i]) & 255u) << (8 * i);
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

// Where a token's slot is: the block of a head, and the token in it.  False if it has none.
__device__ __forceinline__ bool find_slot(const CacheArgs &a, int t, int head, int64_t *block, int *tok)
{
    const int s = a.slots[t];
    if (s < 0)
        return false;
    if ((s >> a.c.page_shift) >= a.c.pages) {
        if (!threadIdx.x || !(threadIdx.x & 7))
            atomicOr(a.flags, LORA_FLAG_CACHE_SLOT);
        return false;
    }
    const int in_page = s & ((1 << a.c.page_shift) - 1);
    *block = cache_block(a.c, s >> a.c.page_shift, head, in_page >> 5);
    *tok = in_page & (kBlock - 1);
    return true;
}

// 8 lanes a token, a lane every eighth unit of 8 dims; 32 tokens a workgroup.
template <typename T, int KIND, int NU>
__global__ __launch_bounds__(256) void cache_store_kernel(CacheArgs a)
{
    typedef Pack<T, 8> P;
    const int t = blockIdx.x * 32 + (threadIdx.x >> 3), head = blockIdx.y, part = threadIdx.x & 7;
    if (t >= a.T)
        return;
    int64_t block;
    int tok;
    if (!find_slot(a, t, head, &block, &tok))
        return;
    const int hd = a.c.head_dim, units = hd >> 3;
    const int64_t from = ((int64_t)t * a.c.kv_heads + head) * hd;
    char *blk = a.c.base + block;
    const bool vec = (((uintptr_t)a.k_in | (uintptr_t)a.v_in) & 15) == 0;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const T *x = (const T *)(side ? a.v_in : a.k_in) + from;
        P p[NU];
        uint32_t high = 0;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = part + 8 * n;
            if (u < units) {
                p[n] = load8(x + 8 * u, vec);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t bits = __float_as_uint(value_of(p[n].v[j])) & 0x7fffffffu;
                    high = bits > high ? bits : high;
                }
            }
        }
        Coding c{};
        if constexpr (KIND != kCacheNative) {
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) {
                const uint32_t o = __shfl_xor(high, d);
                high = o > high ? o : high;
            }
            c = coding_of<KIND>(high);
            if (!part)
                ((float *)(blk + 2 * a.c.half))[side * kBlock + tok] = c.scale;
        }
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = part + 8 * n;
            if (u >= units)
                continue;
            if constexpr (KIND == kCacheNative) {
                if (!side) {
                    *(P *)((T *)blk + key_at(tok, 8 * u)) = p[n];
                } else {
                    T *y = (T *)(blk + a.c.half);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y[value_at(a.c.dp, tok, 8 * u + j)] = p[n].v[j];
                }
            } else {
                float q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    q[j] = c.odd ? 0.f : level_of<KIND>(c, p[n].v[j]);
                const uint2 codes = codes_of<KIND>(q);
                if (!side) {
                    *(uint2 *)(blk + key_at(tok, 8 * u)) = codes;
                } else {
                    uint8_t *y = (uint8_t *)(blk + a.c.half);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y[value_at(a.c.dp, tok, 8 * u + j)] = (uint8_t)((j < 4 ? codes.x : codes.y) >> (8 * (j & 3)));
                }
            }
        }
    }
}

template <typename T, int KIND, int NU>
__global__ __launch_bounds__(256) void cache_load_kernel(CacheArgs a)
{
    typedef Pack<T, 8> P;
    const int t = blockIdx.x * 32 + (threadIdx.x >> 3), head = blockIdx.y, part = threadIdx.x & 7;
    if (t >= a.T)
        return;
    int64_t block;
    int tok;
    if (!find_slot(a, t, head, &block, &tok))
        return;
    const int hd = a.c.head_dim, units = hd >> 3;
    const int64_t to = ((int64_t)t * a.c.kv_heads + head) * hd;
    const char *blk = a.c.base + block;
    const bool vec = (((uintptr_t)a.k_out | (uintptr_t)a.v_out) & 15) == 0;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        T *y = (T *)(side ? a.v_out : a.k_out) + to;
        float scale = 1.f;
        if constexpr (KIND != kCacheNative)
            scale = ((const float *)(blk + 2 * a.c.half))[side * kBlock + tok];
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = part + 8 * n;
            if (u >= units)
                continue;
            P p;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = side ? value_at(a.c.dp, tok, 8 * u + j) : key_at(tok, 8 * u + j);
                if constexpr (KIND == kCacheNative)
                    p.v[j] = ((const T *)(blk + side * a.c.half))[at];
                else
                    put_value(p.v[j], scale * code_value<KIND>(((const uint8_t *)(blk + side * a.c.half))[at]));
            }
            if (vec) {
                *(P *)(y + 8 * u) = p;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[8 * u + j] = p.v[j];
            }
        }
    }
}

template <typename T, int KIND, int NU>
hipError_t launch(bool store, const CacheArgs &a, hipStream_t st)
{
    const dim3 grid((a.T + 31) / 32, a.c.kv_heads);
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
