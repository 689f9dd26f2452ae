// lora_rotary.hip -- gfx950 kernel of rotary positions.
//
//     (a, b) -> amplitude * (a cos w - b sin w, b cos w + a sin w),
//     w = 2 pi * frac(position * turns[pair])
//
// The product and its fraction are taken in double, where a position of 2^31
// still has its angle to 1e-7 of a turn.  Cosine and sine follow from the
// fraction in fp32 for bf16 data (2e-7, far below a bf16 step) and in double for
// fp32 data.
//
// A workgroup owns one token and a share of its heads: it forms the token's
// table of cosines and sines in LDS once, and each thread keeps the entries of
// its piece of a head in registers while it walks the heads.  Bytes bound it:
// 32,556 tokens of 64 heads of 128 (1.07 GB) take 176 us, 6.1 TB/s (a copy of 2 GiB
// reaches 4.85; a third of these bytes fits the last-level cache).  Few tokens take one
// chain, position, angle, sine and cosine, barrier, first load: 512 tokens of 72 heads
// (19 MB) 5.7 us.  Sizes and addresses off 16 bytes go one element at a time (V = 1):
// 8192 tokens of 40 heads of 128 off a boundary 85 us, on it 34; of 40 heads of 80 with 20
// turned 49 us out of place, 19 in place.
#include <hip/hip_runtime.h>

#include "lora_layer.h"

namespace lora {
namespace {

constexpr int kPairs = LORA_ROTARY_MAX_DIM / 2;

template <typename T> struct Elem;
template <> struct Elem<uint16_t> {
    static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t put(float f)
    {
        __bf16 h = (__bf16)f;
        return __builtin_bit_cast(uint16_t, h);
    }
};
template <> struct Elem<float> {
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float f) { return f; }
};

template <typename T, int V> struct alignas(sizeof(T) * V) Pack { T v[V]; };

// V pairs a thread: 16 bytes of each half (HALF), or 16 neighbouring bytes
// (V / 2 pairs); V = 1 is the form without demands on sizes and alignment (one
// pair a thread).
template <typename T, bool HALF, int V>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a)
{
    __shared__ float2 cs[kPairs];
    const int t = blockIdx.x;
    const int pairs = a.rot.rotary_dim >> 1, hd = a.rot.head_dim, rd = a.rot.rotary_dim;
    const double pos = (double)a.positions[t];
    for (int p = threadIdx.x; p < pairs; p += 256) {
        const double turns = pos * a.rot.turns[p];
        const double frac = turns - rint(turns);
        float c, s;
        if constexpr (sizeof(T) == 4) {
            double sd, cd;
            sincospi(2.0 * frac, &sd, &cd);
            c = (float)(cd * a.rot.amplitude);
            s = (float)(sd * a.rot.amplitude);
        } else {
            sincospif(2.f * (float)frac, &s, &c);
            c *= a.rot.amplitude;
            s *= a.rot.amplitude;
        }
        cs[p] = make_float2(c, s);
    }
    __syncthreads();

    // pairs one thread turns, and threads that cover one head
    constexpr int N = V == 1 ? 1 : HALF ? V : V / 2;
    const int pieces = pairs / N;
    const int per_pass = 256 / pieces;            // heads per pass
    const int piece = threadIdx.x % pieces;
    const int first = threadIdx.x / pieces;
    if (first < per_pass) {
        float2 w[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            w[i] = cs[piece * N + i];
        int mi = 0, base = 0;
        for (int h = blockIdx.y * per_pass + first; h < a.total_heads; h += gridDim.y * per_pass) {
            while (h - base >= a.m[mi].heads)
                base += a.m[mi++].heads;
            const int64_t at = (int64_t)t * a.m[mi].width + (int64_t)(h - base) * hd;
            const T *x = (const T *)a.m[mi].x + at;
            T *y = (T *)a.m[mi].y + at;
            if constexpr (V > 1 && HALF) {
                typedef Pack<T, V> P;
                P u = *(const P *)(x + piece * V), v = *(const P *)(x + pairs + piece * V), r, s;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float p = Elem<T>::get(u.v[i]), q = Elem<T>::get(v.v[i]);
                    r.v[i] = Elem<T>::put(fmaf(-q, w[i].y, p * w[i].x));
                    s.v[i] = Elem<T>::put(fmaf(p, w[i].y, q * w[i].x));
                }
                *(P *)(y + piece * V) = r;
                *(P *)(y + pairs + piece * V) = s;
            } else if constexpr (V > 1) {
                typedef Pack<T, V> P;
                P u = *(const P *)(x + piece * V), r;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float p = Elem<T>::get(u.v[2 * i]), q = Elem<T>::get(u.v[2 * i + 1]);
                    r.v[2 * i] = Elem<T>::put(fmaf(-q, w[i].y, p * w[i].x));
                    r.v[2 * i + 1] = Elem<T>::put(fmaf(p, w[i].y, q * w[i].x));
                }
                *(P *)(y + piece * V) = r;
            } else {
                const int i0 = HALF ? piece : 2 * piece, i1 = HALF ? piece + pairs : 2 * piece + 1;
                const float p = Elem<T>::get(x[i0]), q = Elem<T>::get(x[i1]);
                y[i0] = Elem<T>::put(fmaf(-q, w[0].y, p * w[0].x));
                y[i1] = Elem<T>::put(fmaf(p, w[0].y, q * w[0].x));
            }
        }
    }
    // the rest of each head, out of place only
    const int rest = hd - rd;
    if (rest) {
        constexpr int C = V == 1 ? 1 : V;
        const int rp = rest / C;                   // V > 1 asks for whole pieces
        int base = 0;
        for (int mi = 0; mi < a.n; ++mi) {
            const int heads = a.m[mi].heads;
            if (a.m[mi].x != a.m[mi].y) {
                const T *x = (const T *)a.m[mi].x + (int64_t)t * a.m[mi].width;
                T *y = (T *)a.m[mi].y + (int64_t)t * a.m[mi].width;
                for (int i = blockIdx.y * 256 + threadIdx.x; i < heads * rp; i += gridDim.y * 256) {
                    const int at = (i / rp) * hd + rd + (i % rp) * C;
                    if constexpr (V > 1)
                        *(Pack<T, V> *)(y + at) = *(const Pack<T, V> *)(x + at);
                    else
                        y[at] = x[at];
                }
            }
            base += heads;
        }
    }
}

template <typename T, int V>
hipError_t launch(const RotaryArgs &a, hipStream_t st)
{
    const int pairs = a.rot.rotary_dim / 2;
    const bool half = a.rot.layout == LORA_ROTARY_HALF;
    const int pieces = V == 1 ? pairs : half ? pairs / V : pairs / (V / 2);
    const int passes = (a.total_heads + 256 / pieces - 1) / (256 / pieces);
    // enough workgroups for the chip when tokens are few
    const int split = passes < 1 ? 1 : a.T >= 2048 ? 1 : passes < 2048 / a.T ? passes : 2048 / a.T;
    const dim3 grid(a.T, split);
    if (half)
        rotary_kernel<T, true, V><<<grid, 256, 0, st>>>(a);
    else
        rotary_kernel<T, false, V><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(bool bf16, bool vec, const RotaryArgs &a, hipStream_t st)
{
    if (bf16)
        return vec ? launch<uint16_t, 8>(a, st) : launch<uint16_t, 1>(a, st);
    return vec ? launch<float, 4>(a, st) : launch<float, 1>(a, st);
}

}  // namespace lora
