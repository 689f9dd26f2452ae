// lora_norm.hip -- gfx950 kernel of head norms with rotary positions.
//
//     z = x / sqrt(sum x^2 / head_dim + eps) * weight, its pairs turned as lora_rotary.hip turns them
//
// with the sum, the norm and the turn in fp32 and one rounding at the end.  A workgroup owns one
// token and a share of its heads.  A head is cut in items, a pair of 16-byte pieces that turn
// against each other, a piece of neighbouring pairs, or a piece behind rotary_dim; the items go
// to a power of two of neighbouring lanes, which keep them in registers while their sums of
// squares meet in log2 shuffles.  One read and one write of x; for few tokens the chain position, sine
// and cosine, barrier, load, shuffles, store is what it takes.
//
// 64 heads of 128, bf16: 32,556 tokens take 224 us (4.77 TB/s, 0.98 of a copy of 2 GiB), 213 over the same
// tensors again and again, where lora_rotary.hip moves as many bytes in 182: bytes are not all that
// bounds it.  A lane fetches its next head before the sums of this one; the registers for that leave five
// waves a SIMD (rotary positions alone have eight), and more spill (bounds of six 546 us, of eight
// 899).  72 heads, 512 tokens 7.4 us; one token 4.5 us, of which the host's call is 3.4.
#include <hip/hip_runtime.h>

#include "lora_attend.h"

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

// V elements a piece (16 bytes, or 1); NI items a lane.
template <typename T, bool HALF, int V, int NI>
__global__ __launch_bounds__(256) void norm_rotary_kernel(NormArgs a, int lanes)
{
    typedef Pack<T, V> P;
    __shared__ float2 cs[kPairs];
    const RotaryArgs &ro = a.rot;
    const int t = blockIdx.x;
    const int rd = ro.rot.rotary_dim, pairs = rd >> 1, hd = ro.rot.head_dim;
    // Items of a head: `turning` of them hold N pairs each, in one or two pieces, the rest one piece.
    constexpr bool TWO = HALF || V == 1;                 // a turning item has two pieces
    constexpr int N = V == 1 ? 1 : HALF ? V : V / 2;
    const int turning = pairs / N, items = turning + (hd - rd) / V;
    const int per_pass = 256 / lanes, lane = threadIdx.x & (lanes - 1), first = threadIdx.x / lanes;
    int at0[NI], at1[NI];                                // first elements of an item's pieces
    bool turn[NI], used[NI];
#pragma unroll
    for (int k = 0; k < NI; ++k) {
        const int item = lane + k * lanes;
        used[k] = item < items;
        turn[k] = item < turning;
        at0[k] = !turn[k] ? rd + (item - turning) * V : HALF ? item * N : 2 * item * N;
        at1[k] = HALF ? pairs + item * N : 2 * item + 1;
    }
    // A head's values, fetched while the table is formed or the head before is worked on.
    struct Head {
        bool live;
        T *y;
        const T *g;
        P u[NI], v[NI];
    };
    int mi = 0, base = 0;
    auto fetch = [&](int h, Head &s) {
        s.live = h < ro.total_heads;                     // all lanes take part in the shuffles
        while (s.live && h - base >= ro.m[mi].heads)
            base += ro.m[mi++].heads;
        if (!s.live)
            return;
        const int64_t at = (int64_t)t * ro.m[mi].width + (int64_t)(h - base) * hd;
        const T *x = (const T *)ro.m[mi].x + at;
        s.y = (T *)ro.m[mi].y + at;
        s.g = (const T *)a.weight[mi];
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            if (!used[k])
                continue;
            s.u[k] = *(const P *)(x + at0[k]);
            if (TWO && turn[k])
                s.v[k] = *(const P *)(x + at1[k]);
        }
    };
    const int step = gridDim.y * per_pass, h0 = blockIdx.y * per_pass + first;
    Head s;
    fetch(h0, s);

    const double pos = (double)ro.positions[t];
    for (int p = threadIdx.x; p < pairs; p += 256) {
        const double turns = pos * ro.rot.turns[p];
        const double frac = turns - rint(turns);
        float c, s;
        if constexpr (sizeof(T) == 4) {
            double sd, cd;
            sincospi(2.0 * frac, &sd, &cd);
            c = (float)(cd * ro.rot.amplitude);
            s = (float)(sd * ro.rot.amplitude);
        } else {
            sincospif(2.f * (float)frac, &s, &c);
            c *= ro.rot.amplitude;
            s *= ro.rot.amplitude;
        }
        cs[p] = make_float2(c, s);
    }
    __syncthreads();

    float2 w[NI][N];
#pragma unroll
    for (int k = 0; k < NI; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i)
            w[k][i] = turn[k] ? cs[(lane + k * lanes) * N + i] : make_float2(1.f, 0.f);
    const T *loaded = nullptr;                           // the weight in gu and gv
    P gu[NI], gv[NI];
    for (int h = h0 - first; h < ro.total_heads; h += step) {
        Head next;
        fetch(h + first + step, next);
        if (s.live && s.g && s.g != loaded) {
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                if (!used[k])
                    continue;
                gu[k] = *(const P *)(s.g + at0[k]);
                if (TWO && turn[k])
                    gv[k] = *(const P *)(s.g + at1[k]);
            }
            loaded = s.g;
        }
        float sum = 0;
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            if (!s.live || !used[k])
                continue;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float e = Elem<T>::get(s.u[k].v[i]);
                sum = fmaf(e, e, sum);
            }
            if (TWO && turn[k])
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float e = Elem<T>::get(s.v[k].v[i]);
                    sum = fmaf(e, e, sum);
                }
        }
        for (int d = 1; d < lanes; d <<= 1)
            sum += __shfl_xor(sum, d);
        const float r = 1.f / sqrtf(sum / (float)hd + a.eps);
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            if (!s.live || !used[k])
                continue;
            float p[V], q[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                p[i] = Elem<T>::get(s.u[k].v[i]) * r * (s.g ? Elem<T>::get(gu[k].v[i]) : 1.f);
                if (TWO && turn[k])
                    q[i] = Elem<T>::get(s.v[k].v[i]) * r * (s.g ? Elem<T>::get(gv[k].v[i]) : 1.f);
            }
            P out0, out1;
            if (!turn[k]) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    out0.v[i] = Elem<T>::put(p[i]);
            } else if constexpr (TWO) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    out0.v[i] = Elem<T>::put(fmaf(-q[i], w[k][i].y, p[i] * w[k][i].x));
                    out1.v[i] = Elem<T>::put(fmaf(p[i], w[k][i].y, q[i] * w[k][i].x));
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    out0.v[2 * i] = Elem<T>::put(fmaf(-p[2 * i + 1], w[k][i].y, p[2 * i] * w[k][i].x));
                    out0.v[2 * i + 1] = Elem<T>::put(fmaf(p[2 * i], w[k][i].y, p[2 * i + 1] * w[k][i].x));
                }
            }
            *(P *)(s.y + at0[k]) = out0;
            if (TWO && turn[k])
                *(P *)(s.y + at1[k]) = out1;
        }
        s = next;
    }
}

// Where tokens are few, as many workgroups as the chip's 256 CUs hold at once, so that none waits for a
// second round: what the form's registers leave, 4 to 8 a CU.
template <typename T, bool HALF, int V, int NI>
hipError_t launch_items(const NormArgs &a, int lanes, hipStream_t st)
{
    static const int hold = [] {
        int n = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_rotary_kernel<T, HALF, V, NI>, 256, 0) != hipSuccess) {
            (void)hipGetLastError();
            n = 4;
        }
        return 256 * (n < 1 ? 1 : n);
    }();
    const int passes = (a.rot.total_heads + 256 / lanes - 1) / (256 / lanes);
    const int split = passes < hold / a.rot.T ? passes : hold / a.rot.T;
    norm_rotary_kernel<T, HALF, V, NI><<<dim3(a.rot.T, split < 1 ? 1 : split), 256, 0, st>>>(a, lanes);
    return hipGetLastError();
}

template <typename T, bool HALF, int V>
hipError_t launch_half(const NormArgs &a, hipStream_t st)
{
    const lora_rotary &rot = a.rot.rot;
    constexpr int N = V == 1 ? 1 : HALF ? V : V / 2;
    const int items = rot.rotary_dim / 2 / N + (rot.head_dim - rot.rotary_dim) / V;
    int lanes = 1;
    while (lanes < items && lanes < 64)
        lanes *= 2;
    const int each = (items + lanes - 1) / lanes;        // head_dim is at most 512: 1 of 8 elements, 2 of 4, 8 of 1
    static_assert(LORA_NORM_MAX_DIM == 512, "");
    if (each == 1)
        return launch_items<T, HALF, V, 1>(a, lanes, st);
    if constexpr (V < 8)
        if (each == 2)
            return launch_items<T, HALF, V, 2>(a, lanes, st);
    if constexpr (V == 1) {
        if (each <= 4)
            return launch_items<T, HALF, V, 4>(a, lanes, st);
        if (each <= 8)
            return launch_items<T, HALF, V, 8>(a, lanes, st);
    }
    return hipErrorInvalidValue;
}

template <typename T, int V>
hipError_t launch(const NormArgs &a, hipStream_t st)
{
    return a.rot.rot.layout == LORA_ROTARY_HALF ? launch_half<T, true, V>(a, st) : launch_half<T, false, V>(a, st);
}

hipError_t launch_tokens(bool bf16, bool vec, const NormArgs &a, hipStream_t st)
{
    if (bf16)
        return vec ? launch<uint16_t, 8>(a, st) : launch<uint16_t, 1>(a, st);
    return vec ? launch<float, 4>(a, st) : launch<float, 1>(a, st);
}

}  // namespace

hipError_t launch_norm_rotary(bool bf16, bool vec, const NormArgs &a, hipStream_t st)
{
    if (a.rot.T <= kRotaryTokens)
        return launch_tokens(bf16, vec, a, st);
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < a.rot.T && e == hipSuccess; first += kRotaryTokens) {
        NormArgs part = a;
        part.rot = rotary_part(a.rot, first, bf16 ? 2 : 4);
        e = launch_tokens(bf16, vec, part, st);
    }
    return e;
}

}  // namespace lora
