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
// costs accuracy only in the ratio of 16 + q to |q - z|, about two bits of fp32.
// An fp32 x is split into three bf16 numbers (8 + 8 + 8 bits, exact) that are
// multiplied in turn.
//
// An infinity or NaN in x (or an overflow of an intermediate) makes a sum that
// is not finite; such an output is recomputed alone from the formula, so it is
// what plain arithmetic gives.
#include <hip/hip_runtime.h>

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
    const int lane = (int)(i & 63);
    const int64_t block = i >> 6;
    const int kb = (int)(block % KB);
    const int row = (int)(block / KB) * kBaseCols + (lane & 15);
    u32x4 out = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = kb * kBaseK + j * 32 + (lane >> 4) * 8;
        if (row >= a.rows || k >= a.d_in)
            continue;
        const uint32_t w = *(const uint32_t *)(a.q + (int64_t)row * (a.d_in / 2) + k / 2);
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
        // 16 significant bits, to nearest; the freed byte holds 16 + z
        const uint32_t bits = __float_as_uint(s);
        const uint32_t kept = s != s ? 0x7fc00000u : (bits + 0x80u) & 0xffffff00u;
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

// Eight neighbouring inputs of a token as PIECES bf16 operands.
template <typename XT> struct XFrag;
template <> struct XFrag<uint16_t> {
    static constexpr int PIECES = 1;
    bf16x8 p[1];
    __device__ __forceinline__ void load(const uint16_t *src, bool in)
    {
        u32x4 v;
        __builtin_memcpy(&v, src, 16);
        if (!in)
            v = u32x4{0, 0, 0, 0};
        p[0] = __builtin_bit_cast(bf16x8, v);
    }
};
template <> struct XFrag<float> {
    static constexpr int PIECES = 3;
    bf16x8 p[3];
    __device__ __forceinline__ void load(const float *src, bool in)
    {
        float v[8];
        __builtin_memcpy(v, src, 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = in ? v[i] : 0.f;
            const __bf16 hi = (__bf16)f;
            const float r = f - (float)hi;      // exact
            const __bf16 mid = (__bf16)r;
            p[0][i] = hi;
            p[1][i] = mid;
            p[2][i] = (__bf16)(r - (float)mid);
        }
    }
};

template <typename XT>
__device__ __forceinline__ f32x4 mma(const XFrag<XT> &x, bf16x8 w, f32x4 acc)
{
#pragma unroll
    for (int i = XFrag<XT>::PIECES - 1; i >= 0; --i)      // small pieces first
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.p[i], w, acc, 0, 0, 0);
    return acc;
}

__device__ __forceinline__ float activate(float g, int act)
{
    if (act == LORA_ACT_SILU)
        return g / (1.f + expf(-g));
    if (act == LORA_ACT_GELU)      // 1 + erf(v) = erfc(-v), without its cancellation
        return 0.5f * g * erfcf(g * -0.70710678118654752f);
    // (1 + tanh(v)) / 2 = 1 / (1 + exp(-2 v))
    return g / (1.f + expf(-1.59576912160573071f * (g + 0.044715f * g * g * g)));
}

// One output from the formula alone, for sums that are not finite.  x: the
// token's row; q, sc: the column block's first words; n: the column in it.
template <typename XT, int SPB>
__device__ __noinline__ float plain_sum(const XT *x, const uint32_t *q, const typename Scale<XT>::word *sc,
                                        int n, int d_in)
{
    float sum = 0.f;
    for (int k = 0; k < d_in; ++k) {
        const int kb = k >> 7, j = (k >> 5) & 3, g = (k >> 3) & 3, i = k & 7;
        const uint32_t w = q[(int64_t)kb * 256 + (g * 16 + n) * 4 + j];
        const float v = (float)(__builtin_rotateright32(w, 3 + 4 * ((i & 1) * 4 + (i >> 1))) & 15u);
        const typename Scale<XT>::word s = sc[((int64_t)kb * 16 + n) * SPB + ((k & 127) * SPB >> 7)];
        sum += to_f32<XT>(x[k]) * ((v + 16.f - Scale<XT>::zero(s)) * Scale<XT>::scale(s));
    }
    return sum;
}

// ---------------------------------------------------------------------------
// products of few tokens
//
// One workgroup = one block of 16 columns (of gate and of up when GATED) and
// 16 MT tokens; its W waves take the K blocks in turn and join their sums in LDS.
template <typename XT, int MT, int SPB, bool GATED, int W>
__global__ __launch_bounds__(W * 64) void base_few_kernel(BaseArgs a)
{
    typedef typename Scale<XT>::word word;
    constexpr int P = GATED ? 2 : 1;
    // K blocks in flight per wave, by the registers their x takes
    constexpr int U = (sizeof(XT) == 2 ? 4 : 2) / MT > 0 ? (sizeof(XT) == 2 ? 4 : 2) / MT : 1;
    __shared__ float red[W][P][MT][256];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int i = 0;
    if constexpr (!GATED)
        while (i + 1 < a.n && (int)blockIdx.x >= a.col_start[i + 1])
            ++i;
    const BaseMember &m = a.m[i];
    const int nb = blockIdx.x - a.col_start[i];
    const int t0 = blockIdx.y * 16 * MT;
    const int KB = m.kb, d_in = m.d_in;

    const XT *xrow[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        xrow[mt] = (const XT *)m.x + (int64_t)min(t0 + mt * 16 + (lane & 15), a.T - 1) * d_in;
    const uint32_t *q[P];
    const word *sc[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const BaseMember &mp = GATED ? a.m[p] : m;
        q[p] = mp.q + ((int64_t)nb * KB * 64 + lane) * 4;
        sc[p] = (const word *)mp.sc + ((int64_t)nb * KB * 16 + (lane & 15)) * SPB;
    }

    f32x4 tot[P][MT];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            tot[p][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
    const u32x4 ones_bits = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, ones_bits);
    const Constants con = hold_constants();

    for (int kb0 = wave; kb0 < KB; kb0 += W * U) {
        u32x4 wq[U][P];
        word ws[U][P][SPB];
        XFrag<XT> xf[U][MT][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = min(kb0 + u * W, KB - 1);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                wq[u][p] = *(const u32x4 *)(q[p] + (int64_t)kb * 256);
#pragma unroll
                for (int b = 0; b < SPB; ++b)
                    ws[u][p][b] = sc[p][(int64_t)kb * 16 * SPB + b];
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = kb * kBaseK + j * 32 + (lane >> 4) * 8;
                    xf[u][mt][j].load(xrow[mt] + min(k, d_in - 8), k < d_in);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kb0 + u * W >= KB)
                break;
            f32x4 acc[P][MT], sum[MT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if ((j * SPB) % 4 == 0) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        sum[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            acc[p][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
                    }
                }
                bf16x8 b[P];
#pragma unroll
                for (int p = 0; p < P; ++p)
                    b[p] = unpack(wq[u][p][j], con);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        acc[p][mt] = mma<XT>(xf[u][mt][j], b[p], acc[p][mt]);
                    sum[mt] = mma<XT>(xf[u][mt][j], ones, sum[mt]);
                }
                if (((j + 1) * SPB) % 4 == 0) {
                    const int sub = j * SPB / 4;
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const float s = Scale<XT>::scale(ws[u][p][sub]);
                        const float z = Scale<XT>::zero(ws[u][p][sub]);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                tot[p][mt][r] = fmaf(s, fmaf(-z, sum[mt][r], acc[p][mt][r]), tot[p][mt][r]);
                    }
                }
            }
        }
    }

    // lane l holds tokens 4 (l / 16) .. + 3 of column l % 16
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                red[wave][p][mt][((lane >> 4) * 4 + r) * 16 + (lane & 15)] = tot[p][mt][r];
    __syncthreads();
    const int d_out = m.d_out;
    for (int e = threadIdx.x; e < MT * 256; e += W * 64) {
        const int t = t0 + (e >> 4), col = nb * kBaseCols + (e & 15);
        if (t >= a.T || col >= d_out)
            continue;
        float v[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const BaseMember &mp = GATED ? a.m[p] : m;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w)
                s += red[w][p][e >> 8][e & 255];
            if (!(fabsf(s) < __builtin_inff()))
                s = plain_sum<XT, SPB>((const XT *)m.x + (int64_t)t * d_in,
                                       mp.q + (int64_t)nb * KB * 256,
                                       (const word *)mp.sc + (int64_t)nb * KB * 16 * SPB, e & 15, d_in);
            if (mp.bias)
                s += to_f32<XT>(((const XT *)mp.bias)[col]);
            if (mp.add)
                s += to_f32<XT>(((const XT *)mp.add)[(int64_t)t * d_out + col]);
            v[p] = s;
        }
        float out = v[0];
        if constexpr (GATED)
            out = activate(v[0], a.act) * v[P - 1];
        ((XT *)m.y)[(int64_t)t * d_out + col] = from_f32<XT>(out);
    }
}

// ---------------------------------------------------------------------------
// products of many tokens
//
// One workgroup = 16 MT MW tokens x 4 waves of 64 columns (GATED: of 32 of gate
// and the same 32 of up), MW waves above each other.  x is staged in LDS one K
// block at a time and shared by the four column waves; each wave unpacks its own
// weights straight from global memory into the registers its products read.
//
// A group's sum starts at -z' sum x instead of 0, so the zero points cost nothing
// where every column has the same (ZERO false), and one multiplication per sum
// and group where they differ.  The sums of x themselves are formed once per
// workgroup, one K block ahead: wave w multiplies token block w of the next K
// block by ones and leaves the result in LDS.
//
// Block k reads stage k % 3, sums stage (k + 1) % 3 and fills stage (k + 2) % 3,
// which block k - 1 has read; one barrier a block.  16-byte piece p of stage row r
// sits in slot p ^ (r & 15), so the 16 rows of an operand read fall on distinct
// banks.
constexpr int kTileWaveCols = 64;

template <typename XT> struct Staged;      // eight inputs of a token on their way to LDS
template <> struct Staged<uint16_t> {
    u32x4 v;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t src, uint32_t off)
    {
        v = __builtin_amdgcn_raw_buffer_load_b128(src, off, 0, 0);
    }
};
template <> struct Staged<float> {
    float v[8];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t src, uint32_t off)
    {
        const u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(src, off, 0, 0);
        const u32x4 hi = __builtin_amdgcn_raw_buffer_load_b128(src, off, 16, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(lo[i]);
            v[i + 4] = __uint_as_float(hi[i]);
        }
    }
};

template <typename XT, int MT, int MW, int SPB, bool GATED, bool ZERO>
__global__ __launch_bounds__(256 * MW, MW == 1 ? 2 : 1) void base_tile_kernel(BaseArgs a)
{
    typedef typename Scale<XT>::word word;
    constexpr int PIECES = XFrag<XT>::PIECES;
    constexpr int P = GATED ? 2 : 1;
    constexpr int NT = 4;                         // column blocks per wave, gate's first
    constexpr int BM = 16 * MT * MW;
    constexpr int NK = 4 / SPB;                   // MFMA steps per group of a block
    constexpr uint32_t kScBytes = 16 * SPB * sizeof(word);   // scales of a weight block
    __shared__ __attribute__((aligned(16))) uint16_t xs[3][PIECES][BM * kBaseK];
    __shared__ __attribute__((aligned(16))) float sums[2][SPB][BM];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave & 3, wm = wave >> 2;
    const int row = lane & 15, g = lane >> 4;

    // work item -> (column tile, token tile): an XCD takes a contiguous run of items,
    // which go through 8 token tiles of a column tile before the next column tile, so
    // the items it runs together share x and W in its L2
    const int per_xcd = gridDim.x >> 3;
    const int item = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
    if (item >= a.items)
        return;
    const int t_tiles = (a.T + BM - 1) / BM;
    const int c_tiles = a.tile_start[GATED ? 1 : a.n];
    const int band = item / (8 * c_tiles), in = item - band * 8 * c_tiles;
    const int high = min(8, t_tiles - band * 8);
    int c_tile = __builtin_amdgcn_readfirstlane(in / high);
    const int t0 = __builtin_amdgcn_readfirstlane((band * 8 + in - c_tile * high) * BM);
    int mi = 0;
    if constexpr (!GATED)
        while (mi + 1 < a.n && c_tile >= a.tile_start[mi + 1])
            ++mi;
    c_tile -= a.tile_start[mi];
    const BaseMember &m = a.m[mi];
    const int KB = m.kb, d_in = m.d_in, d_out = m.d_out;
    const int nblocks = (d_out + kBaseCols - 1) / kBaseCols;

    // column blocks of this wave (past the last one: that one again, not stored)
    __amdgpu_buffer_rsrc_t q[NT], sc[NT];
    int nb[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int b = GATED ? c_tile * 8 + wn * 2 + (n & 1) : c_tile * 16 + wn * 4 + n;
        nb[n] = b;
        const int64_t at = (int64_t)min(b, nblocks - 1) * KB;
        const BaseMember &mp = GATED ? a.m[n >> 1] : m;
        q[n] = buffer((const char *)mp.q + at * 1024, (uint32_t)KB * 1024u);
        sc[n] = buffer((const char *)mp.sc + at * kScBytes, (uint32_t)KB * kScBytes);
    }
    const uint32_t q_off = lane * 16, sc_off = row * (uint32_t)(SPB * sizeof(word));

    // staging: this thread's piece of MT rows, as offsets from the tile's first row
    const int piece = tid & 15, srow = tid >> 4;
    const uint32_t rows = (uint32_t)min(BM, a.T - t0);
    const auto x0 = buffer((const XT *)m.x + (int64_t)t0 * d_in, rows * (uint32_t)d_in * (uint32_t)sizeof(XT));
    uint32_t src[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        src[i] = (uint32_t)(srow + i * 16 * MW) * (uint32_t)d_in * (uint32_t)sizeof(XT);
    // half of the rows at a time, which is half of the registers
    constexpr int HT = MT / 2;
    Staged<XT> st[HT];
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
            const int r = srow + (half * HT + i) * 16 * MW;
            const int at = r * kBaseK + ((piece ^ (r & 15)) << 3);
            if constexpr (PIECES == 1) {
                *(u32x4 *)&xs[stage][0][at] = st[i].v;
            } else {
                bf16x8 p[3];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float f = st[i].v[e];
                    const __bf16 hi = (__bf16)f;
                    const float rest = f - (float)hi;      // exact
                    const __bf16 mid = (__bf16)rest;
                    p[0][e] = hi;
                    p[1][e] = mid;
                    p[2][e] = (__bf16)(rest - (float)mid);
                }
#pragma unroll
                for (int c = 0; c < PIECES; ++c)
                    *(bf16x8 *)&xs[stage][c][at] = p[c];
            }
        }
    };
    auto x_frag = [&](int stage, int c, int r0, int j) __attribute__((always_inline)) {
        const int r = r0 + row;
        return *(const bf16x8 *)&xs[stage][c][r * kBaseK + (((j * 4 + g) ^ row) << 3)];
    };
    const u32x4 ones_bits = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, ones_bits);
    // -sum x (ZERO) or -24 sum x of this wave's token block, for block kb in `stage`
    auto sum_x = [&](int stage, int kb) __attribute__((always_inline)) {
        if (wn >= MT)
            return;
        const int r0 = (wm * MT + wn) * 16;
#pragma unroll
        for (int sub = 0; sub < SPB; ++sub) {
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = sub * NK; j < (sub + 1) * NK; ++j)
#pragma unroll
                for (int c = PIECES - 1; c >= 0; --c)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x_frag(stage, c, r0, j), ones, acc, 0, 0, 0);
            if (row == 0)
                *(f32x4 *)&sums[kb & 1][sub][r0 + 4 * g] = acc * (ZERO ? -1.f : -24.f);
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
            constexpr int W32 = SPB * (int)sizeof(word) / 4;      // 32-bit words per column
            uint32_t v[W32];
#pragma unroll
            for (int b = 0; b < W32; b += 4) {
                const int off = row * W32 * 4 + b * 4, at = kb * (int)kScBytes;
                if constexpr (W32 == 1) {
                    v[0] = __builtin_amdgcn_raw_buffer_load_b32(sc[n], off, at, 0);
                } else if constexpr (W32 == 2) {
                    const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(sc[n], off, at, 0);
                    v[0] = t[0], v[1] = t[1];
                } else {
                    const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(sc[n], off, at, 0);
                    v[b] = t[0], v[b + 1] = t[1], v[b + 2] = t[2], v[b + 3] = t[3];
                }
            }
            __builtin_memcpy(ws[n], v, sizeof v);
        }
    };
    const Constants con = hold_constants();

    load_w(0);
    // blocks past the last one are read as zeros, staged and never multiplied, so that
    // the loop has no branches
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            load_x(kb, half);
            store_x(kb, half);
        }
    __syncthreads();
    sum_x(0, 0);
    load_x(2, 0);
    __syncthreads();

    int cur = 0;                                  // stage of block k
    for (int k = 0; k < KB; ++k) {
        const int next = cur == 2 ? 0 : cur + 1, fill = next == 2 ? 0 : next + 1;
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
        load_w(min(k + 1, KB - 1));
        store_x(fill, 0);
        load_x(k + 2, 1);
        sum_x(next, k + 1);
        // one group of one token block after the other, its x read a step ahead
        constexpr int STEPS = MT * SPB;
        bf16x8 x[2][NK][PIECES];
        f32x4 c0[2];
        auto read_x = [&](int step) __attribute__((always_inline)) {
            const int r0 = (wm * MT + step / SPB) * 16, sub = step % SPB;
            c0[step & 1] = *(const f32x4 *)&sums[k & 1][sub][r0 + 4 * g];
#pragma unroll
            for (int j = 0; j < NK; ++j)
#pragma unroll
                for (int c = 0; c < PIECES; ++c)
                    x[step & 1][j][c] = x_frag(cur, c, r0, sub * NK + j);
        };
        read_x(0);
#pragma unroll
        for (int step = 0; step < STEPS; ++step) {
            __builtin_amdgcn_sched_barrier(0xf);      // memory operations stay in their step
            const int mt = step / SPB, sub = step % SPB;
            if (step + 1 < STEPS)
                read_x(step + 1);
            if (step == STEPS / 2) {
                store_x(fill, 1);
                load_x(k + 3, 0);
            }
            f32x4 acc[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[n] = ZERO ? c0[step & 1] * z[n][sub] : c0[step & 1];
#pragma unroll
            for (int j = 0; j < NK; ++j)
#pragma unroll
                for (int c = PIECES - 1; c >= 0; --c)
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
        __syncthreads();
        cur = next;
    }

    // lane l holds tokens 4 (l / 16) .. + 3 of column l % 16 of each block
#pragma unroll
    for (int n = 0; n < NT / P; ++n) {
        const int col = nb[n] * kBaseCols + row;
        if (nb[n] >= nblocks || col >= d_out)
            continue;
        float bias[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const BaseMember &mp = GATED ? a.m[p] : m;
            bias[p] = mp.bias ? to_f32<XT>(((const XT *)mp.bias)[col]) : 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = t0 + (wm * MT + mt) * 16 + 4 * g + r;
                if (t >= a.T)
                    continue;
                const int64_t at = (int64_t)t * d_out + col;
                float v[P];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const BaseMember &mp = GATED ? a.m[p] : m;
                    float sum = tot[mt][n + p * (NT / P)][r];
                    if (!(fabsf(sum) < __builtin_inff()))
                        sum = plain_sum<XT, SPB>((const XT *)m.x + (int64_t)t * d_in,
                                                 mp.q + (int64_t)nb[n] * KB * 256,
                                                 (const word *)mp.sc + (int64_t)nb[n] * KB * 16 * SPB,
                                                 row, d_in);
                    if (mp.bias)
                        sum += bias[p];
                    if (mp.add)
                        sum += to_f32<XT>(((const XT *)mp.add)[at]);
                    v[p] = sum;
                }
                float out = v[0];
                if constexpr (GATED)
                    out = activate(v[0], a.act) * v[P - 1];
                ((XT *)m.y)[at] = from_f32<XT>(out);
            }
    }
}

template <typename XT, bool GATED, int SPB, int MT, int MW>
hipError_t launch_tile(const BaseArgs &args, hipStream_t st)
{
    BaseArgs a = args;
    const int cols = GATED ? 8 : 16;              // column blocks of a workgroup
    bool zero = false;
    a.tile_start[0] = 0;
    for (int i = 0; i < a.n; ++i) {
        a.tile_start[i + 1] = a.tile_start[i] + ((a.m[i].d_out + 15) / 16 + cols - 1) / cols;
        zero = zero || a.m[i].zero;
    }
    a.items = a.tile_start[GATED ? 1 : a.n] * ((a.T + 16 * MT * MW - 1) / (16 * MT * MW));
    const int grid = (a.items + 7) / 8 * 8;
    if (zero)
        base_tile_kernel<XT, MT, MW, SPB, GATED, true><<<grid, 256 * MW, 0, st>>>(a);
    else
        base_tile_kernel<XT, MT, MW, SPB, GATED, false><<<grid, 256 * MW, 0, st>>>(a);
    return hipGetLastError();
}

constexpr int kFewTokens = 64;

template <typename XT, bool GATED, int SPB>
hipError_t launch_sized(const BaseArgs &a, hipStream_t st)
{
    const int cols = a.col_start[GATED ? 1 : a.n];
    if (a.T > kFewTokens) {
        if constexpr (sizeof(XT) == 2)
            return launch_tile<XT, GATED, SPB, 4, 1>(a, st);
        else
            return launch_tile<XT, GATED, SPB, 2, 1>(a, st);
    }
    constexpr int W = 8;
    constexpr int MT = sizeof(XT) == 4 || GATED ? 2 : 4;
    if (a.T <= 16)
        base_few_kernel<XT, 1, SPB, GATED, W><<<dim3(cols, 1), W * 64, 0, st>>>(a);
    else
        base_few_kernel<XT, MT, SPB, GATED, W>
            <<<dim3(cols, (a.T + 16 * MT - 1) / (16 * MT)), W * 64, 0, st>>>(a);
    return hipGetLastError();
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
