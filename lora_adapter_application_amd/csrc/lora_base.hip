// lora_base.hip -- gfx950 kernels of the 4-bit base product and its gated form.
//
//     y[t,n] = round( sum_k x[t,k] (q[n,k] - z[n,g]) s[n,g] + bias[n] + add[t,n] ),  g = k / group
//
// The group's factor leaves the sum:
//
//     sum_g s[n,g] ( sum_{k in g} x[t,k] q'[n,k]  -  z'[n,g] sum_{k in g} x[t,k] )
//
// with q' = 16 + q and z' = 16 + z.  q' is a bf16 number whose bits are the
// nibble, shifted, under a constant (16.0 is 0x4180, and q sits in bits 3..6 of
// the mantissa), so a pair of weights costs a shift and one and-or, no weight is
// ever rounded, and the products x q' are exact in the matrix cores' fp32 sums.
// The second sum is the same matrix product with a column of ones.  The offset
// costs accuracy in the ratio of the two sums to their difference: some two bits of
// fp32 where x has no mean, but a sum of 128 inputs near 1 is 3000, and each step that
// rounds it off by up to 2^-13.  bf16 results, off by 2^-9 of their value anyway, do not
// see it.  An fp32 x is split into three bf16 numbers (8 + 8 + 8 bits, exact) that are
// multiplied in turn, and its products keep the large sums short: see base_few_kernel
// and base_tile_kernel.  Their errors in the 2-norm are 0.5e-7 to 4.3e-7, with or without
// a mean (4096 -> 8200: 1 token 1.6e-7 to 2.4e-7, 300 tokens 3.3e-7 to 4.3e-7; a plain
// fp32 product 2.5e-7 to 5.6e-7 and 0.9e-6 to 1.1e-6).
//
// An infinity or NaN in x (or an overflow of an intermediate) makes a sum that
// is not finite; such an output is formed again alone, so it is what plain
// arithmetic gives: infinities and NaNs from their own terms (infinite_sums), the
// rest from the whole formula (plain_sum), which is slow: a batch with an input of
// 3e38 in every row takes 180 times as long as others.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lora_dma.h"
#include "lora_layer.h"

namespace lora {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__device__ __forceinline__ uint16_t f32_to_bf16(float f)
{
    __bf16 h = (__bf16)f;     // round to nearest even
    return __builtin_bit_cast(uint16_t, h);
}

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return f32_to_bf16(v); }
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }

// ---------------------------------------------------------------------------
// repacking, at load time

// One thread per (column block, K block, lane): its 16 bytes of the block from
// four aligned 4-byte reads of its column's row.
__global__ __launch_bounds__(256) void base_pack_q_kernel(BasePackArgs a)
{
    const int KB = (a.d_in + kBaseK - 1) / kBaseK;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t n_items = (int64_t)((a.rows + kBaseCols - 1) / kBaseCols) * KB * 64;
    if (i >= n_items)
        return;
    if (i == 0)
        *a.has_zero = a.zero != nullptr;
    const int lane = (int)(i & 63);
    const int64_t block = i >> 6;
    const int kb = (int)(block % KB);
    const int row = (int)(block / KB) * kBaseCols + (lane & 15);
    u32x4 out = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = kb * kBaseK + j * 32 + (lane >> 4) * 8;
        uint32_t w = 0;
        if (row < a.rows && k < a.d_in) {
            w = *(const uint32_t *)(a.q + (int64_t)row * (a.d_in / 2) + k / 2);
        } else if (row < a.rows) {
            // inputs past d_in: the zero point of their group, so that whatever a kernel
            // multiplies them with cancels
            const int64_t last = (int64_t)row * a.groups + min(k / a.group, a.groups - 1);
            w = (a.zero ? a.zero[last] & 15u : 8u) * 0x11111111u;
        }
        uint32_t r = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r |= ((w >> (8 * e)) & 15u) << (4 * e);               // input 2e
            r |= ((w >> (8 * e + 4)) & 15u) << (4 * (e + 4));     // input 2e + 1
        }
        out[j] = (r << 3) | (r >> 29);
    }
    *(u32x4 *)(a.q_out + i * 4) = out;
}

template <bool BF16>
__global__ __launch_bounds__(256) void base_pack_scale_kernel(BasePackArgs a)
{
    const int KB = (a.d_in + kBaseK - 1) / kBaseK;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t n_items = (int64_t)((a.rows + kBaseCols - 1) / kBaseCols) * KB * kBaseCols * a.spb;
    if (i >= n_items)
        return;
    const int sub = (int)(i % a.spb);
    const int64_t j = i / a.spb;
    const int n = (int)(j & 15);
    const int64_t block = j >> 4;
    const int k = (int)(block % KB) * kBaseK + sub * (kBaseK / a.spb);
    const int row = (int)(block / KB) * kBaseCols + n;
    float s = 0.f;
    uint32_t z = 8;
    if (row < a.rows && k < a.d_in) {
        const int64_t at = (int64_t)row * a.groups + k / a.group;
        s = a.scale[at];
        if (a.zero)
            z = a.zero[at] & 15u;
    }
    if constexpr (BF16) {
        // 16 significant bits, to nearest, so that a scale and its zero point are one word of
        // 4 bytes: off by 2^-16 of a normal number at most, where a bf16 result is rounded by
        // 2^-9 to 2^-8.  The freed byte holds 16 + z
        const uint32_t bits = __float_as_uint(s);
        uint32_t kept = (bits + 0x80u) & 0xffffff00u;
        if (s != s)
            kept = 0x7fc00000u;
        else if ((kept & 0x7fffffffu) == 0x7f800000u)
            kept = bits & 0xffffff00u;             // the largest numbers stay finite
        ((uint32_t *)a.sc_out)[i] = kept | (16u + z);
    } else {
        ((float2 *)a.sc_out)[i] = make_float2(s, 16.f + (float)z);
    }
}

// ---------------------------------------------------------------------------
// pieces of the products

// `bytes` bytes from a wave-uniform address as a buffer: a load of it takes its
// address from scalar registers and one 32-bit offset, and reads 0 past the end.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, uint32_t bytes)
{
    const uint64_t at = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)((uint64_t)hi << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

// The eight weights of a word as bf16 numbers 16 + q.  mask and one are 0x00780078
// and 0x41804180 in registers (hold_constants): as literals the and and the or would
// be two instructions.
struct Constants {
    uint32_t mask, one;
};
__device__ __forceinline__ Constants hold_constants()
{
    Constants c = {0x00780078u, 0x41804180u};
    asm("" : "+s"(c.mask));
    asm("" : "+v"(c.one));
    return c;
}
__device__ __forceinline__ bf16x8 unpack(uint32_t w, const Constants &c)
{
    u32x4 r;
    r[0] = (w & c.mask) | c.one;
    r[1] = ((w >> 4) & c.mask) | c.one;
    r[2] = ((w >> 8) & c.mask) | c.one;
    r[3] = (__builtin_rotateright32(w, 12) & c.mask) | c.one;
    return __builtin_bit_cast(bf16x8, r);
}

// The eight weights of a word as bf16 numbers q - z, exact, at three instructions a weight:
// sums of their products are the formula's own.
__device__ __forceinline__ bf16x8 unpack_exact(uint32_t w, float z)
{
    const uint32_t r = __builtin_rotateright32(w, 3);
    const uint32_t half[2] = {r & 0x0f0f0f0fu, (r >> 4) & 0x0f0f0f0fu};
    bf16x8 out;
#pragma unroll
    for (int i = 0; i < 8; ++i)                   // input i: nibble i / 2 + 4 (i % 2)
        out[i] = (__bf16)((float)((half[(i >> 1) & 1] >> (16 * (i & 1) + 8 * (i >> 2))) & 255u) - z);
    return out;
}

template <typename XT> struct Scale;
template <> struct Scale<uint16_t> {
    typedef uint32_t word;
    static __device__ __forceinline__ float scale(word w) { return __uint_as_float(w & 0xffffff00u); }
    static __device__ __forceinline__ float zero(word w) { return (float)(w & 0xffu); }
};
template <> struct Scale<float> {
    typedef float2 word;
    static __device__ __forceinline__ float scale(word w) { return w.x; }
    static __device__ __forceinline__ float zero(word w) { return w.y; }
};

// bf16 numbers that an input is split into.
template <typename XT> constexpr int XT_PIECES = sizeof(XT) == 2 ? 1 : 3;

__device__ __forceinline__ float activate(float g, int act)
{
    if (act == LORA_ACT_SILU)
        return g / (1.f + expf(-g));
    if (act == LORA_ACT_GELU)      // 1 + erf(v) = erfc(-v), without its cancellation
        return 0.5f * g * erfcf(g * -0.70710678118654752f);
    // (1 + tanh(v)) / 2 = 1 / (1 + exp(-2 v))
    return g / (1.f + expf(-1.59576912160573071f * (g + 0.044715f * g * g * g)));
}

// The terms x W of one input and four neighbouring columns, added to v.  q, sc: the column
// block's first words; n: the first of the columns in it.
template <typename XT, int SPB>
__device__ __forceinline__ void add_terms(f32x4 &v, float x, const uint32_t *q, const typename Scale<XT>::word *sc,
                                          int n, int k)
{
    const int kb = k >> 7, j = (k >> 5) & 3, g = (k >> 3) & 3, i = k & 7;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t w = __builtin_rotateright32(q[(int64_t)kb * 256 + (g * 16 + n + c) * 4 + j], 3);
        const typename Scale<XT>::word sw = sc[((int64_t)kb * 16 + n + c) * SPB + ((k & 127) * SPB >> 7)];
        v[c] += x * (((float)((w >> (4 * ((i & 1) * 4 + (i >> 1)))) & 15u) - (Scale<XT>::zero(sw) - 16.f)) *
                     Scale<XT>::scale(sw));
    }
}

// Four neighbouring outputs of a row with infinities or NaNs in it: their terms decide, where
// the others can neither overflow nor be infinite themselves (inputs that add up to less than
// 2^60 and scales below it: 15 * 2^120 at most).  Else, or without such an input, zeros.  So
// a batch with an infinity in every row costs a scan of its rows for every four outputs (1024
// tokens of 4096 -> 4096 764 us, and with whole sums 7800; without infinities 46).
template <typename XT, int SPB>
__device__ __noinline__ f32x4 infinite_sums(const XT *x, const uint32_t *q, const typename Scale<XT>::word *sc,
                                            int n, int d_in)
{
    constexpr float kSmall = 1.15292150460684698e18f;    // 2^60
    const float inf = __builtin_inff();
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    float rest = 0.f;                             // sum of the other inputs' sizes
    for (int k = 0; k < d_in; k += 32) {          // four loads in flight
        XT e[32];
#pragma unroll
        for (int u = 0; u < 32; u += 8)           // past d_in: the row's last eight again
            __builtin_memcpy(e + u, x + min(k + u, d_in - 8), 8 * sizeof(XT));
        float size = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            size += fabsf(to_f32<XT>(e[i]));
        if (size < inf) {
            rest += size;
            continue;
        }
        for (int i = 0; i < min(32, d_in - k); ++i) {
            const float f = to_f32<XT>(x[k + i]);
            if (fabsf(f) < inf)
                rest += fabsf(f);
            else
                add_terms<XT, SPB>(v, f, q, sc, n, k + i);
        }
        if (v[0] != v[0] && v[1] != v[1] && v[2] != v[2] && v[3] != v[3])
            return v;                             // nothing changes a NaN
    }
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    if (!(rest < kSmall))
        return none;
    for (int kb = 0; kb < (d_in + kBaseK - 1) / kBaseK; ++kb)
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int b = 0; b < SPB; ++b)
                if (!(fabsf(Scale<XT>::scale(sc[((int64_t)kb * 16 + n + c) * SPB + b])) < kSmall))
                    return none;
    return v;                                     // 0 in no place, or in all
}

// One output from the formula alone, for the other sums that are not finite.  x: the
// token's row; q, sc: the column block's first words; n: the column in it.
template <typename XT, int SPB>
__device__ __noinline__ float plain_sum(const XT *x, const uint32_t *q, const typename Scale<XT>::word *sc,
                                        int n, int d_in)
{
    float sum = 0.f;
    for (int k = 0; k < d_in && sum == sum; k += 8) {
        const int kb = k >> 7, j = (k >> 5) & 3, g = (k >> 3) & 3;
        const uint32_t w = __builtin_rotateright32(q[(int64_t)kb * 256 + (g * 16 + n) * 4 + j], 3);
        const typename Scale<XT>::word sw = sc[((int64_t)kb * 16 + n) * SPB + ((k & 127) * SPB >> 7)];
        const float s = Scale<XT>::scale(sw), z = Scale<XT>::zero(sw) - 16.f;
        XT v[8];
        __builtin_memcpy(v, x + k, sizeof v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum += to_f32<XT>(v[i]) * (((float)((w >> (4 * ((i & 1) * 4 + (i >> 1)))) & 15u) - z) * s);
    }
    return sum;
}

// Four neighbouring outputs of a token from their sums v[weight]: bias, add, the
// activation, and one rounding.
template <typename XT, int SPB, bool GATED>
__device__ __forceinline__ void finish(const BaseArgs &a, int mi, const f32x4 *v, int t, int col)
{
    constexpr int P = GATED ? 2 : 1;
    const BaseMember &m = a.m[mi];
    const int64_t at = (int64_t)t * m.d_out + col;
    f32x4 f[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const BaseMember &mp = a.m[GATED ? p : mi];
        f[p] = v[p];
        XT e[4];
        if (mp.bias) {
            __builtin_memcpy(e, (const XT *)mp.bias + col, sizeof e);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[p][i] += to_f32<XT>(e[i]);
        }
        if (mp.add) {
            __builtin_memcpy(e, (const XT *)mp.add + at, sizeof e);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[p][i] += to_f32<XT>(e[i]);
        }
    }
    XT out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = from_f32<XT>(GATED ? activate(f[0][i], a.act) * f[P - 1][i] : f[0][i]);
    __builtin_memcpy((XT *)m.y + at, out, sizeof out);
}

// finish() where every sum is finite; else false, and nothing is stored.
template <typename XT, int SPB, bool GATED>
__device__ __forceinline__ bool finish_finite(const BaseArgs &a, int mi, const f32x4 *v, int t, int col)
{
    float big = 0.f;
#pragma unroll
    for (int p = 0; p < (GATED ? 2 : 1); ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            big += fabsf(v[p][i]);                // infinite or NaN as any of them is
    if (!(big < __builtin_inff()))
        return false;
    finish<XT, SPB, GATED>(a, mi, v, t, col);
    return true;
}

// finish() with the four sums formed again from the formula.
template <typename XT, int SPB, bool GATED>
__device__ __forceinline__ void finish_again(const BaseArgs &a, int mi, int t, int col)
{
    typedef typename Scale<XT>::word word;
    const BaseMember &m = a.m[mi];
    const int64_t block = (int64_t)(col >> 4) * m.kb;
    f32x4 v[2];
#pragma unroll
    for (int p = 0; p < (GATED ? 2 : 1); ++p) {
        const BaseMember &mp = a.m[GATED ? p : mi];
        const XT *x = (const XT *)m.x + (int64_t)t * m.d_in;
        const uint32_t *q = mp.q + block * 256;
        const word *sc = (const word *)mp.sc + block * (16 * SPB);
        v[p] = infinite_sums<XT, SPB>(x, q, sc, col & 15, m.d_in);
        if (v[p][0] != 0.f)
            continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[p][i] = plain_sum<XT, SPB>(x, q, sc, (col & 15) + i, m.d_in);
    }
    finish<XT, SPB, GATED>(a, mi, v, t, col);
}

// ---------------------------------------------------------------------------
// products of few tokens
//
// One workgroup = C blocks of 16 columns (of gate and of up when GATED) and
// 16 MT tokens; its W waves take the K blocks in turn and join their sums in LDS.
// Each wave keeps D blocks in flight.  Bytes bound it: one token through q, k and v of
// 4096 -> 4096 (27 MB) takes 7.1 us, gate and up of 4096 -> 11008 (49 MB) 10.9 us, 3.8
// and 4.5 TB/s with the launch and the first load's latency in it.  With more tokens
// the bytes of x count, which every workgroup reads whole: see launch_sized.
//
// fp32 (see the top): two token blocks multiply q - z itself (EXACT), whose unpacking two
// blocks share; one token block joins the sums after every 32 inputs, where each is rounded
// once at its full size, since the small pieces of x come first (4096 -> 4096: 24 tokens
// 16.4 us against 17.0 with sums of a whole group, 64 tokens 33.8 / 34.3; one token of
// 4096 -> 4096 8.8 / 8.5, 5120 -> 10240 14.8 / 14.3, gated 4096 -> 11008 21.1 / 18.9, and
// 27 with q - z).
template <typename XT> struct RawX;        // eight inputs of a token as they were loaded
template <> struct RawX<uint16_t> {
    u32x4 v;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t src, uint32_t off)
    {
        v = __builtin_amdgcn_raw_buffer_load_b128(src, off, 0, 0);
    }
    __device__ __forceinline__ void split(bf16x8 *p) const { p[0] = __builtin_bit_cast(bf16x8, v); }
};
template <> struct RawX<float> {
    u32x4 v[2];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t src, uint32_t off)
    {
        v[0] = __builtin_amdgcn_raw_buffer_load_b128(src, off, 0, 0);
        v[1] = __builtin_amdgcn_raw_buffer_load_b128(src, off + 16, 0, 0);
    }
    __device__ __forceinline__ void split(bf16x8 *p) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = __uint_as_float(v[i >> 2][i & 3]);
            const __bf16 hi = (__bf16)f;
            const float rest = f - (float)hi;      // exact
            const __bf16 mid = (__bf16)rest;
            p[0][i] = hi;
            p[1][i] = mid;
            p[2][i] = (__bf16)(rest - (float)mid);
        }
    }
};

// The scale words of one column and K block, off + at bytes into the buffer (at is
// wave-uniform and inside it).
template <typename XT, int SPB>
__device__ __forceinline__ void load_scales(typename Scale<XT>::word *out, __amdgpu_buffer_rsrc_t src,
                                            uint32_t off, uint32_t at)
{
    constexpr int W32 = SPB * (int)sizeof(typename Scale<XT>::word) / 4;
    uint32_t v[W32];
    if constexpr (W32 == 1) {
        v[0] = __builtin_amdgcn_raw_buffer_load_b32(src, off, at, 0);
    } else if constexpr (W32 == 2) {
        const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(src, off, at, 0);
        v[0] = t[0], v[1] = t[1];
    } else {
#pragma unroll
        for (int b = 0; b < W32; b += 4) {
            const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(src, off + b * 4, at, 0);
            v[b] = t[0], v[b + 1] = t[1], v[b + 2] = t[2], v[b + 3] = t[3];
        }
    }
    __builtin_memcpy(out, v, sizeof v);
}

// Whether the weights of member mi (gated: either weight) were loaded with zero points, from
// the word that the load wrote (kZerosAsk).
template <bool GATED>
__device__ __forceinline__ bool has_zero(const BaseArgs &a, int mi)
{
    const uint32_t z = GATED ? *a.m[0].has_zero | *a.m[1].has_zero : *a.m[mi].has_zero;
    return __builtin_amdgcn_readfirstlane(z) != 0;
}

// Column tiles of `width` columns of each member; returns how many there are.
template <bool GATED>
int set_tiles(BaseArgs &a, int width)
{
    a.tile_start[0] = 0;
    for (int i = 0; i < a.n; ++i)
        a.tile_start[i + 1] = a.tile_start[i] + (a.m[i].d_out + width - 1) / width;
    return a.tile_start[GATED ? 1 : a.n];
}

template <typename XT, int MT, int C, int SPB, bool GATED, int W, int D>
__global__ __launch_bounds__(W * 64) void base_few_kernel(BaseArgs a)
{
    typedef typename Scale<XT>::word word;
    constexpr int PIECES = XT_PIECES<XT>;
    constexpr int P = GATED ? 2 : 1;
    constexpr int B = P * C;                      // weight blocks, each weight's C together
    constexpr bool EXACT = PIECES > 1 && MT > 1;  // products of q - z, without sums of x
    constexpr int JOINS = PIECES > 1 && !EXACT ? 4 : SPB;    // of the sums of a block
    constexpr int PG = JOINS > SPB && B > 4 ? 4 : B;         // weight blocks whose sums are held at once
    constexpr uint32_t kScBytes = 16 * SPB * sizeof(word);
    __shared__ __attribute__((aligned(16))) float red[W][B][MT][256];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, g = lane >> 4;
    int i = 0;
    if constexpr (!GATED)
        while (i + 1 < a.n && (int)blockIdx.x >= a.tile_start[i + 1])
            ++i;
    const BaseMember &m = a.m[i];
    const int nb = (blockIdx.x - a.tile_start[i]) * C;
    const int t0 = blockIdx.y * 16 * MT;
    const int KB = m.kb, d_in = m.d_in;

    // tokens past the batch read 0
    const uint32_t x_row = (uint32_t)d_in * (uint32_t)sizeof(XT);
    const auto xb = buffer((const XT *)m.x + (int64_t)t0 * d_in, (uint32_t)min(16 * MT, a.T - t0) * x_row);
    uint32_t x_off[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        x_off[mt] = (uint32_t)(mt * 16 + row) * x_row + g * 8 * (uint32_t)sizeof(XT);
    const int nblocks = (m.d_out + kBaseCols - 1) / kBaseCols;
    __amdgpu_buffer_rsrc_t q[B], sc[B];
#pragma unroll
    for (int p = 0; p < B; ++p) {                 // past the last block: that one again, not stored
        const BaseMember &mp = GATED ? a.m[p / C] : m;
        const int64_t at = (int64_t)min(nb + p % C, nblocks - 1) * KB;
        q[p] = buffer((const char *)mp.q + at * 1024, (uint32_t)KB * 1024u);
        sc[p] = buffer((const char *)mp.sc + at * kScBytes, (uint32_t)KB * kScBytes);
    }

    u32x4 wq[D][B];
    word ws[D][B][SPB];
    RawX<XT> xr[D][MT][4];
    // Blocks past the last one lie past the ends of the weights' buffers and read zeros;
    // inputs past d_in are sent past the end of x's.  The whole offset is the lanes'
    // own: a scalar offset past the end of a buffer is not checked against it.
    auto load = [&](int d, int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < B; ++p) {
            wq[d][p] = __builtin_amdgcn_raw_buffer_load_b128(q[p], (uint32_t)kb * 1024u + lane * 16, 0, 0);
            load_scales<XT, SPB>(ws[d][p], sc[p], (uint32_t)kb * kScBytes + row * (uint32_t)(SPB * sizeof(word)), 0);
        }
        const int left = d_in - kb * kBaseK;
        const uint32_t at = (uint32_t)kb * (uint32_t)(kBaseK * sizeof(XT));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                xr[d][mt][j].load(xb, j * 32 + g * 8 < left ? x_off[mt] + at + j * 32 * (uint32_t)sizeof(XT)
                                                            : 0x80000000u);
    };

    f32x4 tot[B][MT];
#pragma unroll
    for (int p = 0; p < B; ++p)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            tot[p][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
    const u32x4 ones_bits = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, ones_bits);
    const Constants con = hold_constants();

#pragma unroll
    for (int d = 0; d < D; ++d)
        load(d, wave + d * W);
    for (int kb0 = wave; kb0 < KB; kb0 += D * W) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (kb0 + d * W >= KB)
                break;
            f32x4 acc[B][MT], sum[MT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if ((j * JOINS) % 4 == 0) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        sum[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int p = 0; p < B; ++p)
                            acc[p][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
                    }
                }
#pragma unroll
                for (int p0 = 0; p0 < B; p0 += PG) {
                    bf16x8 b[PG];
#pragma unroll
                    for (int p = 0; p < PG; ++p) {
                        uint32_t q8 = wq[d][p0 + p][j];
                        if constexpr (PG < B)         // in its turn
                            asm volatile("" : "+v"(q8));
                        b[p] = EXACT ? unpack_exact(q8, Scale<XT>::zero(ws[d][p0 + p][j * SPB / 4]) - 16.f)
                                     : unpack(q8, con);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        bf16x8 x[PIECES];
                        xr[d][mt][j].split(x);
#pragma unroll
                        for (int c = PIECES - 1; c >= 0; --c) {      // small pieces first
#pragma unroll
                            for (int p = 0; p < PG; ++p)
                                acc[p0 + p][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[c], b[p], acc[p0 + p][mt],
                                                                                          0, 0, 0);
                            if (!EXACT && p0 == 0)
                                sum[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[c], ones, sum[mt], 0, 0, 0);
                        }
                    }
                    if (((j + 1) * JOINS) % 4 == 0) {
                        const int sub = j * SPB / 4;
#pragma unroll
                        for (int p = p0; p < p0 + PG; ++p) {
                            const float s = Scale<XT>::scale(ws[d][p][sub]);
                            const float z = Scale<XT>::zero(ws[d][p][sub]);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    tot[p][mt][r] = fmaf(s, EXACT ? acc[p][mt][r]
                                                                  : fmaf(-z, sum[mt][r], acc[p][mt][r]),
                                                         tot[p][mt][r]);
                                // joined here, not behind the next block's loads, which need the registers
                                if constexpr (JOINS > SPB)
                                    asm volatile("" : "+v"(tot[p][mt]));
                            }
                        }
                    }
                }
            }
            if (kb0 + (d + D) * W < KB)
                load(d, kb0 + (d + D) * W);
        }
    }

    // lane l holds tokens 4 (l / 16) .. + 3 of column l % 16
#pragma unroll
    for (int p = 0; p < B; ++p)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                red[wave][p][mt][(g * 4 + r) * 16 + row] = tot[p][mt][r];
    __syncthreads();
    for (int e = threadIdx.x; e < C * MT * 64; e += W * 64) {
        const int c = e / (MT * 64), in = e % (MT * 64) * 4;
        const int t = t0 + (in >> 4), col = (nb + c) * kBaseCols + (in & 15);
        if (t >= a.T || col >= m.d_out)
            continue;
        f32x4 v[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            v[p] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < W; ++w)
                v[p] += *(const f32x4 *)&red[w][p * C + c][in >> 8][in & 255];
        }
        if (!finish_finite<XT, SPB, GATED>(a, i, v, t, col))
            finish_again<XT, SPB, GATED>(a, i, t, col);
    }
}

template <typename XT, int MT, int C, int SPB, bool GATED, int W, int D>
hipError_t launch_few(const BaseArgs &args, hipStream_t st)
{
    BaseArgs a = args;
    const int cols = set_tiles<GATED>(a, 16 * C);
    base_few_kernel<XT, MT, C, SPB, GATED, W, D><<<dim3(cols, (a.T + 16 * MT - 1) / (16 * MT)), W * 64, 0, st>>>(a);
    return hipGetLastError();
}

// Work item -> (member, its column tile, the first token of its token tile): an XCD takes a
// contiguous run of items, which go through 8 token tiles of a column tile before the next
// column tile, so the items it runs together share x and W in its L2.  False: no item.
template <bool GATED, int BM>
__device__ __forceinline__ bool item_of(const BaseArgs &a, int &mi, int &c_tile, int &t0)
{
    const int per_xcd = gridDim.x >> 3;
    const int item = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
    if (item >= a.items)
        return false;
    const int t_tiles = (a.T + BM - 1) / BM;
    const int c_tiles = a.tile_start[GATED ? 1 : a.n];
    const int band = item / (8 * c_tiles), in = item - band * 8 * c_tiles;
    const int high = min(8, t_tiles - band * 8);
    c_tile = __builtin_amdgcn_readfirstlane(in / high);
    t0 = __builtin_amdgcn_readfirstlane((band * 8 + in - c_tile * high) * BM);
    mi = 0;
    if constexpr (!GATED)
        while (mi + 1 < a.n && c_tile >= a.tile_start[mi + 1])
            ++mi;
    c_tile -= a.tile_start[mi];
    return true;
}

// ---------------------------------------------------------------------------
// products of many tokens
//
// One workgroup = 16 MT tokens x 4 waves of 16 NT columns (GATED: half of them
// gate's, half the same columns of up), in KW groups of four waves that take the K
// blocks in turn and join their sums in LDS.  x is staged in LDS one K block at a
// time and shared by the four column waves, by direct-to-LDS loads where x lies on a
// 16-byte boundary (DX), else through registers; each wave unpacks its own weights
// from global memory into the registers its products read, so a weight is unpacked
// once per 16 MT tokens.
//
// A group's sum starts at -z' sum x instead of 0, so the zero points cost nothing
// where every column has the same (ZERO false), and one multiplication per sum
// and group where they differ.  The sums of x themselves are formed once per
// workgroup, one K block ahead: wave w multiplies token block w of the next K
// block by ones and leaves the result in LDS.
//
// Block k reads stage k % 3, sums stage (k + 1) % 3 and fills stage (k + 2) % 3,
// which block k - 1 has read; one barrier a block, before its last products.  16-byte
// piece p of stage row r sits in slot p ^ (r & 15), so the 16 rows of an operand read
// fall on distinct banks.
//
// bf16 takes 64 x 256 tiles (MT = NT = 4), whose 64 fp32 sums, 64 registers of
// unpacked weights and two steps of x fill the 256 registers of two waves a SIMD: two
// workgroups a CU, each under the other's waits.  Groups of 32 with zero points spill 3
// to 6 of them, and x through registers 4 to 16.  Measured on 8192 tokens: 4096 -> 4096
// with a residual 302 us (909 TFLOP/s), gated 4096 -> 11008 1495 us (988 TFLOP/s; a
// library's bf16 product of 8192^3 reaches 1375 on the same card).  The matrix cores
// are busy half of the time, and the vector unit, which unpacks, scales and also issues
// the matrix instructions, 0.7 of it.  One workgroup of eight waves on 128 x 256 with
// weights in LDS too was slower (1642 against 1562 us then).
template <typename XT, int MT, int NT, int KW, int SPB, bool GATED> struct TileLds {
    static constexpr int P = GATED ? 2 : 1;
    static constexpr int BM = 16 * MT, BN = 64 * (NT / P);
    static constexpr int RN = BN + 4;             // row of joined sums, padded for the banks
    static constexpr size_t kStageBytes = (size_t)KW * 3 * XT_PIECES<XT> * BM * kBaseK * 2;
    static constexpr size_t kJoinBytes = (size_t)KW * P * (BM / 2) * RN * 4;
    __attribute__((aligned(16))) unsigned char stages[kStageBytes > kJoinBytes ? kStageBytes : kJoinBytes];
    __attribute__((aligned(16))) float sums[KW][2][SPB][BM];
    __attribute__((aligned(16))) float unread[256 + 2 * SPB * BM];
};

template <typename XT, int MT, int NT, int KW, int SPB, bool GATED, bool ZERO, bool DX>
__device__ __forceinline__ void base_tile(const BaseArgs &a, TileLds<XT, MT, NT, KW, SPB, GATED> &shared,
                                          int mi, int c_tile, int t0)
{
    typedef typename Scale<XT>::word word;
    constexpr int PIECES = XT_PIECES<XT>;
    constexpr int P = GATED ? 2 : 1;
    constexpr int NP = NT / P;                    // column blocks per wave and weight
    constexpr int BM = 16 * MT, BN = 64 * NP;
    constexpr int NK = 4 / SPB;                   // MFMA steps per group of a block
    constexpr uint32_t kScBytes = 16 * SPB * sizeof(word);   // scales of a weight block
    constexpr int RN = std::remove_reference_t<decltype(shared)>::RN;
    unsigned char *const lds = shared.stages;
    auto &unread = shared.unread;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave & 3, kg = wave >> 2;
    const int tid = threadIdx.x & 255;            // in its group
    auto &xs = ((uint16_t(*)[3][PIECES][BM * kBaseK])lds)[kg];
    auto &sums = shared.sums[kg];
    const int row = lane & 15, g = lane >> 4;

    const BaseMember &m = a.m[mi];
    const int KB = m.kb, d_in = m.d_in, d_out = m.d_out;
    const int nblocks = (d_out + kBaseCols - 1) / kBaseCols;

    // column blocks of this wave (past the last one: that one again, not stored)
    __amdgpu_buffer_rsrc_t q[NT], sc[NT];
    int nb[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int b = (c_tile * 4 + wn) * NP + n % NP;
        nb[n] = b;
        const int64_t at = (int64_t)min(b, nblocks - 1) * KB;
        const BaseMember &mp = GATED ? a.m[n / NP] : m;
        q[n] = buffer((const char *)mp.q + at * 1024, (uint32_t)KB * 1024u);
        sc[n] = buffer((const char *)mp.sc + at * kScBytes, (uint32_t)KB * kScBytes);
    }

    // staging: this thread's piece of MT rows, as offsets from the tile's first row
    const int piece = tid & 15, srow = tid >> 4;
    const uint32_t rows = (uint32_t)min(BM, a.T - t0);
    const auto x0 = buffer((const XT *)m.x + (int64_t)t0 * d_in, rows * (uint32_t)d_in * (uint32_t)sizeof(XT));
    uint32_t src[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        src[i] = (uint32_t)(srow + i * 16) * (uint32_t)d_in * (uint32_t)sizeof(XT);
    // half of the rows at a time, which is half of the registers
    constexpr int HT = MT / 2;
    RawX<XT> st[HT];
    auto load_x = [&](int kb, int half) __attribute__((always_inline)) {
        const int k = kb * kBaseK + piece * 8;
        // inputs past d_in read 0, as rows past the batch do: an offset past the buffer
        const uint32_t at = k < d_in ? (uint32_t)k * (uint32_t)sizeof(XT) : 0x80000000u;
#pragma unroll
        for (int i = 0; i < HT; ++i)
            st[i].load(x0, src[half * HT + i] + at);
    };
    auto store_x = [&](int stage, int half) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < HT; ++i) {
            const int r = srow + (half * HT + i) * 16;
            const int at = r * kBaseK + ((piece ^ (r & 15)) << 3);
            bf16x8 p[PIECES];
            st[i].split(p);
#pragma unroll
            for (int c = 0; c < PIECES; ++c)
                *(bf16x8 *)&xs[stage][c][at] = p[c];
        }
    };
    // or, with direct-to-LDS loads (DX): MT of them a wave and block, 4 rows each; rows
    // past the batch and inputs past d_in repeat the last (weights past d_in equal their
    // zero point, so those products cancel)
    const char *xd = (const char *)m.x + (int64_t)t0 * d_in * 2;
    const uint32_t xs_at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) unsigned char *)lds +
                           (uint32_t)(kg * 3 * PIECES * BM * kBaseK * 2);
    uint32_t xd_row[MT], xd_k[MT];
#pragma unroll
    for (int i = 0; DX && i < MT; ++i) {
        const int r = 4 * (wn + 4 * i) + (lane >> 4);
        xd_row[i] = (uint32_t)min(r, a.T - 1 - t0) * (uint32_t)d_in * 2u;
        xd_k[i] = (uint32_t)(((lane & 15) ^ (r & 15)) * 8);
    }
    auto dma_x = [&](int stage, int kb) __attribute__((always_inline)) {
        const uint32_t at = xs_at + (uint32_t)(stage * BM * kBaseK * 2 + wn * 1024);
        if ((kb + 1) * kBaseK <= d_in) {          // a whole block: its place in the rows is scalar
#pragma unroll
            for (int i = 0; i < MT; ++i)
                dma16_off(xd + (int64_t)kb * (kBaseK * 2), xd_row[i] + xd_k[i] * 2u, at + (uint32_t)(i * 4096));
        } else {
#pragma unroll
            for (int i = 0; i < MT; ++i)
                dma16_off(xd, xd_row[i] + min((uint32_t)kb * kBaseK + xd_k[i], (uint32_t)d_in - 8u) * 2u,
                          at + (uint32_t)(i * 4096));
        }
    };
    // every load is in, every read of LDS done, in every wave
    auto landed = [&]() __attribute__((always_inline)) {
        if constexpr (DX)
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        else
            __syncthreads();
    };
    auto x_frag = [&](int stage, int c, int r0, int j) __attribute__((always_inline)) {
        const int r = r0 + row;
        return *(const bf16x8 *)&xs[stage][c][r * kBaseK + (((j * 4 + g) ^ row) << 3)];
    };
    const u32x4 ones_bits = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, ones_bits);
    // -sum x (ZERO) or -24 sum x of this wave's token block, for block kb in `stage`.
    // Every column of the product is the sum: the lanes of column 0 store it, the others
    // store to a place that nobody reads, which costs less than a branch.
    float *const sum_at = row == 0 ? &sums[0][0][wn * 16 + 4 * g] : &unread[lane * 4];
    auto store_sum = [&](f32x4 acc, int kb, int sub) __attribute__((always_inline)) {
        *(f32x4 *)(sum_at + ((kb & 1) * SPB + sub) * BM) = acc * (ZERO ? -1.f : -24.f);
    };
    auto sum_x = [&](int stage, int kb) __attribute__((always_inline)) {
        if (wn >= MT)
            return;
#pragma unroll
        for (int sub = 0; sub < SPB; ++sub) {
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = PIECES - 1; c >= 0; --c)          // small pieces first
#pragma unroll
                for (int j = sub * NK; j < (sub + 1) * NK; ++j)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x_frag(stage, c, wn * 16, j), ones, acc, 0, 0, 0);
            store_sum(acc, kb, sub);
        }
    };
    f32x4 tot[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            tot[mt][n] = f32x4{0.f, 0.f, 0.f, 0.f};

    u32x4 wq[NT];
    word ws[NT][SPB];
    auto load_w = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            wq[n] = __builtin_amdgcn_raw_buffer_load_b128(q[n], lane * 16, kb * 1024, 0);
            load_scales<XT, SPB>(ws[n], sc[n], row * (uint32_t)(SPB * sizeof(word)), (uint32_t)kb * kScBytes);
        }
    };
    const Constants con = hold_constants();

    // this group's block k is block k KW + kg of the weights; blocks past the last one
    // repeat it against inputs of 0
    const int nk = (KB + KW - 1) / KW;
    auto w_block = [&](int k) __attribute__((always_inline)) { return min(k * KW + kg, KB - 1); };

    load_w(w_block(0));
    // blocks past the last one are staged too (as zeros, or with DX the rows' last inputs
    // again) and never multiplied, so that the loop has no branches
    if constexpr (DX) {
        dma_x(0, kg);
        dma_x(1, KW + kg);
    } else {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                load_x(kb * KW + kg, half);
                store_x(kb, half);
            }
    }
    landed();
    sum_x(0, 0);
    if constexpr (!DX)
        load_x(2 * KW + kg, 0);
    landed();

    constexpr int STEPS = MT * SPB;
    static_assert(STEPS % 2 == 0, "x alternates between two sets of registers");
    bf16x8 x[2][NK][PIECES];
    f32x4 c0[2];
    auto read_x = [&](int stage, int k, int step) __attribute__((always_inline)) {
        const int r0 = step / SPB * 16, sub = step % SPB;
        c0[step & 1] = *(const f32x4 *)&sums[k & 1][sub][r0 + 4 * g];
#pragma unroll
        for (int c = 0; c < PIECES; ++c)
#pragma unroll
            for (int j = 0; j < NK; ++j)
                x[step & 1][j][c] = x_frag(stage, c, r0, sub * NK + j);
    };
    read_x(0, 0, 0);
    int cur = 0;                                  // stage of block k
    for (int k = 0; k < nk; ++k) {
        const int next = cur == 2 ? 0 : cur + 1, fill = next == 2 ? 0 : next + 1;
        if constexpr (DX) {
            // the weights' wait, here where it is over and before further loads start
#pragma unroll
            for (int n = 0; n < NT; ++n)
                asm volatile("" : "+v"(wq[n]), "+v"(ws[n][0]));
            dma_x(fill, (k + 2) * KW + kg);
        }
        bf16x8 w[NT][4];
        float s[NT][SPB], z[NT][SPB];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[n][j] = unpack(wq[n][j], con);
#pragma unroll
            for (int b = 0; b < SPB; ++b) {
                s[n][b] = Scale<XT>::scale(ws[n][b]);
                z[n][b] = ZERO ? Scale<XT>::zero(ws[n][b]) : 0.f;
            }
        }
        load_w(w_block(k + 1));
        if constexpr (!DX) {
            store_x(fill, 0);
            load_x((k + 2) * KW + kg, 1);
        }
        sum_x(next, k + 1);
        // one group of one token block after the other, its x read a step ahead; before the
        // last one's products, when this block has been read, the waves meet, and the next
        // block's first x is read under those products
#pragma unroll
        for (int step = 0; step < STEPS; ++step) {
            // nothing moves between the steps, nor the reads behind the products: left alone,
            // the reads sink to where they are waited for (8192 tokens of 4096 -> 4096: 296
            // against 289 us; groups of 32, 2048 tokens of 5120 -> 10240: 399 against 349)
            // (fp32, whose steps hold three times the x, keeps to the order of its reads only)
            constexpr int FREE = PIECES == 1 ? 0 : 0xf;
            __builtin_amdgcn_sched_barrier(FREE);
            const int mt = step / SPB, sub = step % SPB;
            if (!DX && step == STEPS / 2) {
                store_x(fill, 1);
                load_x((k + 3) * KW + kg, 0);
            }
            if (step + 1 < STEPS) {
                read_x(cur, k, step + 1);
            } else {
                landed();
                read_x(next, k + 1, 0);
            }
            if constexpr (PIECES == 1)
                __builtin_amdgcn_sched_barrier(0);
            f32x4 acc[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[n] = ZERO ? c0[step & 1] * z[n][sub] : c0[step & 1];
            // large pieces first (fp32): they bring the sum down from -z' sum x, and the others
            // are added to what is small then.  With the pieces of each step together twelve
            // steps a group round a large sum, not four: 2.5 times the error, 1.5 to 4% faster
#pragma unroll
            for (int c = 0; c < PIECES; ++c)
#pragma unroll
                for (int j = 0; j < NK; ++j)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[step & 1][j][c], w[n][sub * NK + j],
                                                                         acc[n], 0, 0, 0);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    tot[mt][n][r] = fmaf(s[n][sub], acc[n][r], tot[mt][n][r]);
        }
        cur = next;
    }

    // Through LDS, so that y is written (and add read) in rows: in two halves of the
    // tokens, which fit the stages.  Lane l holds tokens 4 (l / 16) .. + 3 of column
    // l % 16 of each block.
    float *red = (float *)lds;                    // [KW][P][BM / 2][RN]
    constexpr int PASSES = (BM / 2 * BN / 4 + 256 * KW - 1) / (256 * KW);
    static_assert(2 * PASSES <= 32, "a bit for each of a thread's fours");
    uint32_t again = 0;                           // fours with a sum that is not finite
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        landed();                                 // the last reads of the stages, or of the first half
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int mt = 0; mt < MT / 2; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    red[((kg * P + n / NP) * (BM / 2) + mt * 16 + 4 * g + r) * RN + (wn * NP + n % NP) * 16 + row] =
                        tot[half * (MT / 2) + mt][n][r];
        __syncthreads();
#pragma unroll
        for (int pass = 0; pass < PASSES; ++pass) {
            const int e = threadIdx.x + pass * (256 * KW);
            const int r = e / (BN / 4), c = e % (BN / 4) * 4;
            const int t = t0 + half * (BM / 2) + r, col = c_tile * BN + c;
            if (e >= BM / 2 * BN / 4 || t >= a.T || col >= d_out)
                continue;
            f32x4 v[P];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                v[p] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < KW; ++w)
                    v[p] += *(const f32x4 *)&red[((w * P + p) * (BM / 2) + r) * RN + c];
            }
            if (!finish_finite<XT, SPB, GATED>(a, mi, v, t, col))
                again |= 1u << (half * PASSES + pass);
        }
    }
    // behind the sums' last use, so that the call costs the rest no registers
    while (again) {
        const int bit = __builtin_ctz(again);
        again &= again - 1;
        const int e = threadIdx.x + bit % PASSES * (256 * KW);
        finish_again<XT, SPB, GATED>(a, mi, t0 + bit / PASSES * (BM / 2) + e / (BN / 4),
                                     c_tile * BN + e % (BN / 4) * 4);
    }
}

template <typename XT, int MT, int NT, int KW, int SPB, bool GATED, bool DX, Zeros Z>
__global__ __launch_bounds__(256 * KW, KW == 1 ? 2 : 1) void base_tile_kernel(BaseArgs a)
{
    __shared__ TileLds<XT, MT, NT, KW, SPB, GATED> shared;
    int mi, c_tile, t0;
    if (!item_of<GATED, 16 * MT>(a, mi, c_tile, t0))
        return;
    if (Z == kZerosSome || (Z == kZerosAsk && has_zero<GATED>(a, mi)))
        base_tile<XT, MT, NT, KW, SPB, GATED, true, DX>(a, shared, mi, c_tile, t0);
    else
        base_tile<XT, MT, NT, KW, SPB, GATED, false, DX>(a, shared, mi, c_tile, t0);
}

// ---------------------------------------------------------------------------
// products of a middling number of tokens
//
// bf16, x on a 16-byte boundary, too few tiles to fill the chip: a workgroup of
// 16 MT tokens x CW waves of 16 NT columns splits the K blocks over KW groups of waves,
// and x, weights and scales are all brought to LDS by direct-to-LDS loads, S - 1 blocks
// ahead and without registers.  Each wave forms the sums of x of all its rows itself,
// in the block they belong to.  24 tokens of 11008 -> 4096 take 15.8 us (few-token
// kernel 19.4), 64 tokens of gated 4096 -> 11008 23.0 (54).  Per K block of a group the
// LDS reads, the unpacking and a chain of products follow each other: that latency,
// times the blocks of a group, is the time.  So LDS goes to groups before stages: with 2
// stages of more groups in place of 3 or 4 of 2 groups, 100 tokens of 11008 -> 11008 take
// 48.2 us (51.8), 64 tokens of it 33.8 (35.4), and 64 tokens of 4096 -> 11008 in groups of
// 32 19.4 (22.7).  The 32 x 32 tiles, whose 4 groups are small, keep 3 stages, and so do
// the 32 x 64 where there is one scale a block; the largest, 64 x 384 on 8 waves of 48
// columns, fill LDS with one group of 3 (4 waves of 96 columns, one a SIMD: 512 tokens of
// 5120 -> 10240 86.5 us against 68.5).  A wave takes NT weight blocks in a row of gate's
// and then up's, so it may have blocks of one only.
// Without zero points the products start at -24 sum x, which halves the vector work per
// sum but waits for that sum first: 512 tokens of 5120 -> 10240 in groups of 64 84 -> 74
// us, gated 256 tokens 63 -> 60, 64 tokens of 4096 -> 11008 in groups of 32 19.1 -> 17.3;
// the smallest grids, which wait most, gain nothing or lose a little (64 tokens of 4096 ->
// 4096 8.8 us with zero points and 8.9 without, of gated 4096 -> 11008 23.0 and 23.4).
//
// Block k of a group lies in stage k % S; block k + S - 1 is loaded into the stage of
// block k - 1 once every wave has read that.  Every wave issues the same number of loads
// a block (LOADS), so the wait that lets the last S - 2 blocks' loads stand is a constant.
// Rows past the batch, inputs past d_in and blocks past the last one are addressed inside
// the buffers and drop out: such rows are not stored, such inputs have weights equal to
// their zero point, and such blocks get scale 0.
template <int MT, int NT, int CW, int KW, int S, int SPB, bool GATED> struct SplitLds {
    static constexpr int P = GATED ? 2 : 1, WB = CW * NT, BM = 16 * MT;
    static constexpr int kStage = BM * kBaseK * 2 + WB * 1024 + (WB * SPB + 3) / 4 * 256;   // of a group
    static constexpr int RN = 16 * (WB / P) + 4;
    static constexpr int kJoin = KW * P * BM * RN * 4;
    __attribute__((aligned(16))) unsigned char bytes[S * kStage * KW > kJoin ? S * kStage * KW : kJoin];
};

template <int MT, int NT, int CW, int KW, int S, int SPB, bool GATED, bool ZERO>
__device__ __forceinline__ void base_split(const BaseArgs &a, SplitLds<MT, NT, CW, KW, S, SPB, GATED> &shared,
                                           int mi, int c_tile, int t0)
{
    constexpr int P = GATED ? 2 : 1;
    constexpr int WB = CW * NT;                   // weight blocks of a workgroup, gate's before up's
    constexpr int CB = WB / P;                    // column blocks: wave w multiplies weight blocks NT w ..
    constexpr int BM = 16 * MT, BN = 16 * CB;
    constexpr int NK = 4 / SPB;
    constexpr int XL = BM / 4 / CW;               // loads of x a wave and block
    constexpr int kX = BM * kBaseK * 2, kW = WB * 1024, SL = (WB * SPB + 3) / 4, kS = SL * 256;
    constexpr int kStage = kX + kW + kS;          // LDS bytes of a group's stage
    typedef std::remove_reference_t<decltype(shared)> Lds;
    static_assert(kStage == Lds::kStage, "");
    constexpr int RN = Lds::RN;
    constexpr int SW = (SL + CW - 1) / CW;        // scale loads (SL of 256 bytes a block) of each wave
    constexpr int LOADS = XL + NT + SW;
    static_assert(WB % P == 0 && BM / 4 % CW == 0, "");
    static_assert(!GATED || CB * SPB % 4 == 0, "a load of scales is of one weight");
    static_assert((S - 2) * LOADS < 64, "vmcnt counts to 63");
    unsigned char *const lds = shared.bytes;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = wave / CW, wn = wave % CW;
    const int row = lane & 15, g = lane >> 4;

    const BaseMember &m = a.m[mi];
    const int KB = m.kb, d_in = m.d_in, d_out = m.d_out;
    const int nblocks = (d_out + kBaseCols - 1) / kBaseCols;
    const int nk = (KB + KW - 1) / KW;

    unsigned char *const my = lds + kg * S * kStage;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) unsigned char *)my;

    // this wave's loads of a block: XL of x (4 rows of 256 bytes each), NT weight blocks,
    // and its share of the scales (where there are fewer, several waves load the same)
    const char *x0 = (const char *)m.x + (int64_t)t0 * d_in * 2;
    uint32_t x_row[XL], x_k[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int r = 4 * (wn + CW * i) + (lane >> 4);
        x_row[i] = (uint32_t)min(r, a.T - 1 - t0) * (uint32_t)d_in * 2u;
        x_k[i] = (uint32_t)(((lane & 15) ^ (r & 15)) * 8);
    }
    // weight block b of the workgroup: weight b / CB, column block b % CB
    auto block_at = [&](int b) __attribute__((always_inline)) {
        return (int64_t)min(c_tile * CB + b % CB, nblocks - 1) * KB;
    };
    const char *wsrc[NT], *ssrc[SW];
    uint32_t s_off[SW], s_at[SW];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int b = wn + CW * i;
        wsrc[i] = (const char *)(GATED ? a.m[b / CB] : m).q + block_at(b) * 1024;
    }
#pragma unroll
    for (int i = 0; i < SW; ++i) {
        const int l = min(wn + CW * i, SL - 1);
        const int word = min(l * 64 + lane, WB * 16 * SPB - 1);   // word of the workgroup's scales
        const int b = word / (16 * SPB);
        const int b0 = l * 64 / (16 * SPB);       // the load's first block: all are of one weight
        ssrc[i] = (const char *)(GATED ? a.m[b0 / CB] : m).sc + block_at(b0) * (16 * SPB * 4);
        s_off[i] = (uint32_t)((block_at(b) - block_at(b0)) * (16 * SPB) + word % (16 * SPB)) * 4u;
        s_at[i] = (uint32_t)(kX + kW + l * 256);
    }
    auto load = [&](int stage, int k) __attribute__((always_inline)) {
        const int kb = min(k * KW + kg, KB - 1);
        const uint32_t at = lds0 + (uint32_t)(stage * kStage);
#pragma unroll
        for (int i = 0; i < XL; ++i)
            dma16_off(x0, x_row[i] + min((uint32_t)kb * kBaseK + x_k[i], (uint32_t)d_in - 8u) * 2u,
                      at + (uint32_t)((wn + CW * i) * 1024));
#pragma unroll
        for (int i = 0; i < NT; ++i)
            dma16_off(wsrc[i] + (int64_t)kb * 1024, lane * 16, at + (uint32_t)(kX + (wn + CW * i) * 1024));
#pragma unroll
        for (int i = 0; i < SW; ++i)
            dma4_off(ssrc[i] + (int64_t)kb * (16 * SPB * 4), s_off[i], at + s_at[i]);
    };
    auto landed = [&]() __attribute__((always_inline)) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * LOADS) : "memory");
    };
    // ones, or -24 where that is every zero point: then the products start at -24 sum x
    constexpr uint32_t kOne = ZERO ? 0x3f803f80u : 0xc1c0c1c0u;
    const u32x4 ones_bits = {kOne, kOne, kOne, kOne};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, ones_bits);
    const Constants con = hold_constants();

    f32x4 tot[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            tot[mt][n] = f32x4{0.f, 0.f, 0.f, 0.f};

#pragma unroll
    for (int k = 0; k < S - 1; ++k)
        load(k, k);
    landed();

    // Before the products of a block's last step, when the wave has read all it needs of
    // the block, it meets the others, and reads the weights and first x of the next block
    // under those products.
    constexpr int STEPS = MT * SPB;
    static_assert(STEPS % 2 == 0, "x alternates between two sets of registers");
    u32x4 raw[NT];
    uint32_t sw[NT][SPB];
    bf16x8 x[2][NK];
    auto read_w = [&](const unsigned char *st) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int b = wn * NT + n;
            raw[n] = *(const u32x4 *)(st + kX + b * 1024 + lane * 16);
#pragma unroll
            for (int i = 0; i < SPB; ++i)
                sw[n][i] = ((const uint32_t *)(st + kX + kW))[(b * 16 + row) * SPB + i];
        }
    };
    auto read_x = [&](const unsigned char *st, int step) __attribute__((always_inline)) {
        const int r0 = step / SPB * 16, sub = step % SPB;
#pragma unroll
        for (int j = 0; j < NK; ++j)
            x[step & 1][j] = *(const bf16x8 *)(st + (r0 + row) * 256 + ((((sub * NK + j) * 4 + g) ^ row) << 4));
    };
    read_w(my);
    read_x(my, 0);
    int cur = 0;
    for (int k = 0; k < nk; ++k) {
        load(cur == 0 ? S - 1 : cur - 1, k + S - 1);
        const unsigned char *st = my + cur * kStage;
        cur = cur == S - 1 ? 0 : cur + 1;
        bf16x8 w[NT][4];
        float s[NT][SPB], z[NT][SPB];
        const bool dead = k * KW + kg >= KB;      // a block past the last one
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[n][j] = unpack(raw[n][j], con);
#pragma unroll
            for (int i = 0; i < SPB; ++i) {
                s[n][i] = dead ? 0.f : Scale<uint16_t>::scale(sw[n][i]);
                z[n][i] = ZERO ? Scale<uint16_t>::zero(sw[n][i]) : 0.f;
            }
        }
#pragma unroll
        for (int step = 0; step < STEPS; ++step) {
            // memory operations stay in their step (with short steps everything does)
            __builtin_amdgcn_sched_barrier(SPB == 1 ? 0xf : 0);
            const int mt = step / SPB, sub = step % SPB;
            if (step + 1 < STEPS) {
                read_x(st, step + 1);
            } else {
                landed();
                read_w(my + cur * kStage);
                read_x(my + cur * kStage, 0);
            }
            f32x4 acc[NT], sum = {0.f, 0.f, 0.f, 0.f};
            if constexpr (!ZERO)
#pragma unroll
                for (int j = 0; j < NK; ++j)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[step & 1][j], ones, sum, 0, 0, 0);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[n] = ZERO ? f32x4{0.f, 0.f, 0.f, 0.f} : sum;
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                if constexpr (ZERO)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[step & 1][j], ones, sum, 0, 0, 0);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[step & 1][j], w[n][sub * NK + j], acc[n],
                                                                     0, 0, 0);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    tot[mt][n][r] = fmaf(s[n][sub], ZERO ? fmaf(-z[n][sub], sum[r], acc[n][r]) : acc[n][r],
                                         tot[mt][n][r]);
        }
    }
    // the loads of blocks past the last one are in before the stages hold sums
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

    // lane l holds tokens 4 (l / 16) .. + 3 of column l % 16 of each block
    float *red = (float *)lds;                // [KW][P][BM][RN]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int b = wn * NT + n;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                red[((kg * P + b / CB) * BM + mt * 16 + 4 * g + r) * RN + b % CB * 16 + row] = tot[mt][n][r];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < BM * BN / 4; e += 64 * CW * KW) {
        const int r = e / (BN / 4), c = e % (BN / 4) * 4;
        const int t = t0 + r, col = c_tile * BN + c;
        if (t >= a.T || col >= d_out)
            continue;
        f32x4 v[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            v[p] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < KW; ++w)
                v[p] += *(const f32x4 *)&red[((w * P + p) * BM + r) * RN + c];
        }
        if (!finish_finite<uint16_t, SPB, GATED>(a, mi, v, t, col))
            finish_again<uint16_t, SPB, GATED>(a, mi, t, col);
    }
}

template <int MT, int NT, int CW, int KW, int S, int SPB, bool GATED, Zeros Z>
__global__ __launch_bounds__(64 * CW * KW) void base_split_kernel(BaseArgs a)
{
    __shared__ SplitLds<MT, NT, CW, KW, S, SPB, GATED> shared;
    int mi, c_tile, t0;
    if (!item_of<GATED, 16 * MT>(a, mi, c_tile, t0))
        return;
    if (Z == kZerosSome || (Z == kZerosAsk && has_zero<GATED>(a, mi)))
        base_split<MT, NT, CW, KW, S, SPB, GATED, true>(a, shared, mi, c_tile, t0);
    else
        base_split<MT, NT, CW, KW, S, SPB, GATED, false>(a, shared, mi, c_tile, t0);
}

template <typename F> void with_zeros(Zeros zeros, F &&launch)
{
    switch (zeros) {
    case kZerosNone: launch(std::integral_constant<Zeros, kZerosNone>{}); break;
    case kZerosSome: launch(std::integral_constant<Zeros, kZerosSome>{}); break;
    default: launch(std::integral_constant<Zeros, kZerosAsk>{});
    }
}

template <bool GATED, int SPB, int MT, int NT, int CW, int KW, int S>
hipError_t launch_split(const BaseArgs &args, hipStream_t st)
{
    BaseArgs a = args;
    constexpr int BM = 16 * MT, BN = 16 * CW * NT / (GATED ? 2 : 1);
    a.items = set_tiles<GATED>(a, BN) * ((a.T + BM - 1) / BM);
    const int grid = (a.items + 7) / 8 * 8;
    with_zeros(a.zeros, [&](auto z) {
        base_split_kernel<MT, NT, CW, KW, S, SPB, GATED, z.value><<<grid, 64 * CW * KW, 0, st>>>(a);
    });
    return hipGetLastError();
}

template <typename XT, bool GATED, int SPB, int MT, int NT, int KW, bool DX>
hipError_t launch_tile(const BaseArgs &args, hipStream_t st)
{
    BaseArgs a = args;
    constexpr int BM = 16 * MT, BN = 64 * (GATED ? NT / 2 : NT);
    a.items = set_tiles<GATED>(a, BN) * ((a.T + BM - 1) / BM);
    const int grid = (a.items + 7) / 8 * 8;
    with_zeros(a.zeros, [&](auto z) {
        base_tile_kernel<XT, MT, NT, KW, SPB, GATED, DX, z.value><<<grid, 256 * KW, 0, st>>>(a);
    });
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// which kernel

constexpr int kCus = 256;

// Whether tiles of BM tokens and BN columns are at most one per CU.
template <bool GATED>
bool one_per_cu(const BaseArgs &args, int BM, int BN)
{
    BaseArgs a = args;
    return (int64_t)set_tiles<GATED>(a, BN) * ((a.T + BM - 1) / BM) <= kCus;
}

// Up to 16 tokens the weights' bytes decide and one MFMA row block holds the batch.
// A workgroup of one column block reads all of x for 16 columns; where there are two
// blocks a CU or more, workgroups of C = 4 blocks read a quarter of that (microseconds,
// bf16, 5120 -> 10240: 1 token 8.3 against 8.5, 4 tokens 10.2 / 8.6, 16 tokens
// 17.1 / 9.4; gated 4096 -> 11008, whose two weights share x already: 8 tokens
// 12.2 / 12.2, 16 tokens 15.8 / 13.0; fp32, which also splits x into bf16 pieces less
// often: 1 token of 5120 -> 10240 21.8 / 14.8).  With fewer blocks they would leave CUs
// idle (4096 -> 4096, 16 tokens: 6.5 / 7.8).  Groups of 32 keep four scales a block: two
// column blocks of gate and of up are what the registers hold.
//
// Above that, the smallest tile of which every CU gets at most one, since such a batch
// waits for its slowest workgroup (4096 -> 4096: 64 tokens 8.6 us on 32 x 32, 10.5 on
// 32 x 64, 14.6 on 32 x 128 tiles; 256 tokens 27.7, 22.5, 18.1; 5120 -> 10240, 256
// tokens: 54 on 64 x 128, 43 on 64 x 256; 512 tokens 78 on 64 x 256, some CUs with two,
// and 68.5 on 64 x 384); with more, the tile kernel, two workgroups a CU (8192 tokens of
// 4096 -> 4096: 292 us against 345 on the 64 x 384 split).
// x off a 16-byte boundary cannot be loaded to LDS directly and takes slower ways.
template <typename XT, bool GATED, int SPB>
hipError_t launch_sized(const BaseArgs &a, hipStream_t st)
{
    constexpr bool WIDE = sizeof(XT) == 4;
    int blocks = 0;
    bool aligned = true;
    for (int i = 0; i < (GATED ? 1 : a.n); ++i) {
        blocks += (a.m[i].d_out + kBaseCols - 1) / kBaseCols;
        aligned = aligned && ((uintptr_t)a.m[i].x & 15) == 0;
    }
    if (a.T <= 16) {
        if (blocks >= 2 * kCus && (WIDE || a.T > (GATED ? 8 : 2)))
            return launch_few<XT, 1, GATED && SPB == 4 ? 2 : 4, SPB, GATED, 8, 1>(a, st);
        // (gate and up in flight together: one token of 4096 -> 11008 10.9 us, 11.4 with two each)
        return launch_few<XT, 1, 1, SPB, GATED, 8, GATED && !WIDE ? 1 : 2>(a, st);
    }
    if constexpr (WIDE) {
        // (24 tokens: 4096 -> 4096 16.4 us against 34, 5120 -> 10240 51 against 42; 128 tokens
        // of 1000 -> 1296 9.4 against 12.0, 256 tokens 13.1 against 12.4)
        if ((int64_t)blocks * ((a.T + 31) / 32) <= 2 * kCus)
            return launch_few<XT, 2, 1, SPB, GATED, 8, 1>(a, st);
        if (one_per_cu<GATED>(a, 32, GATED ? 64 : 128))
            return launch_tile<XT, GATED, SPB, 2, 2, 2, false>(a, st);
        return launch_tile<XT, GATED, SPB, 2, 4, 1, false>(a, st);
    } else {
        if (!aligned)
            return a.T <= 64 ? launch_few<XT, 2, 1, SPB, GATED, 8, 2>(a, st)
                             : launch_tile<XT, GATED, SPB, 4, 4, 1, false>(a, st);
        if constexpr (GATED) {
            if (one_per_cu<true>(a, 32, 64))
                return launch_split<true, SPB, 2, 2, 4, 4, 2>(a, st);
            if (one_per_cu<true>(a, 64, 64))
                return launch_split<true, SPB, 4, 2, 4, 3, 2>(a, st);
            if (one_per_cu<true>(a, 64, 128))
                return launch_split<true, SPB, 4, 4, 4, 2, 2>(a, st);
            if (one_per_cu<true>(a, 64, 192))
                return launch_split<true, SPB, 4, 3, 8, 1, 3>(a, st);
        } else {
            if (one_per_cu<false>(a, 32, 32))
                return launch_split<false, SPB, 2, 1, 2, 4, 3>(a, st);
            if (one_per_cu<false>(a, 32, 64))
                return launch_split<false, SPB, 2, 1, 4, 4, SPB == 1 ? 3 : 2>(a, st);
            if (one_per_cu<false>(a, 32, 128))
                return launch_split<false, SPB, 2, 2, 4, 4, 2>(a, st);
            if (one_per_cu<false>(a, 64, 128))
                return launch_split<false, SPB, 4, 2, 4, 3, 2>(a, st);
            if (one_per_cu<false>(a, 64, 256))
                return launch_split<false, SPB, 4, 4, 4, 2, 2>(a, st);
            if (one_per_cu<false>(a, 64, 384))
                return launch_split<false, SPB, 4, 3, 8, 1, 3>(a, st);
        }
        return launch_tile<XT, GATED, SPB, 4, 4, 1, true>(a, st);
    }
}

template <typename XT, bool GATED>
hipError_t launch_spb(int spb, const BaseArgs &a, hipStream_t st)
{
    switch (spb) {
    case 1: return launch_sized<XT, GATED, 1>(a, st);
    case 2: return launch_sized<XT, GATED, 2>(a, st);
    default: return launch_sized<XT, GATED, 4>(a, st);
    }
}

}  // namespace

hipError_t launch_base_pack(bool bf16, const BasePackArgs &a, hipStream_t st)
{
    const int64_t KB = (a.d_in + kBaseK - 1) / kBaseK;
    const int64_t blocks = (int64_t)((a.rows + kBaseCols - 1) / kBaseCols) * KB;
    const unsigned gq = (unsigned)((blocks * 64 + 255) / 256);
    const unsigned gs = (unsigned)((blocks * kBaseCols * a.spb + 255) / 256);
    base_pack_q_kernel<<<gq, 256, 0, st>>>(a);
    if (bf16)
        base_pack_scale_kernel<true><<<gs, 256, 0, st>>>(a);
    else
        base_pack_scale_kernel<false><<<gs, 256, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_base(bool bf16, bool gated, int spb, const BaseArgs &a, hipStream_t st)
{
    if (bf16)
        return gated ? launch_spb<uint16_t, true>(spb, a, st) : launch_spb<uint16_t, false>(spb, a, st);
    return gated ? launch_spb<float, true>(spb, a, st) : launch_spb<float, false>(spb, a, st);
}

}  // namespace lora
