// Device helpers of the linear-attention kernels.
#pragma once

#include "la.h"

namespace ss {
namespace la {

template <typename T> __device__ __forceinline__ float ldf(const T* p);
template <> __device__ __forceinline__ float ldf<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float ldf<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <> __device__ __forceinline__ float ldf<__half>(const __half* p) { return __half2float(*p); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;
// Smallest log decay taken as it is: e^-128 is zero in f32 already, and a
// bounded value keeps differences of cumulative decays finite (g = -inf).
constexpr float kMinG = -128.0f;

__device__ __forceinline__ float clamp_g(float g) { return g < kMinG ? kMinG : g; }  // keeps NaN

__device__ __forceinline__ int64_t row_length(const Args& a, int64_t b) {
    if (!a.lengths) return a.L;
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : (n > a.L ? a.L : n);
}

__device__ __forceinline__ float log_decay(const Args& a, int64_t b, int64_t t, int64_t h) {
    return clamp_g(a.g_per_head ? a.g[h] : a.g[(b * a.L + t) * a.H + h]);
}

// A decay e^g of an f32 state: S + (e^g - 1) S where it is weak (a rounded e^g near 1
// would be off the same way at every step, which a long memory adds up), e^g S below
// one half (e^g - 1 is next to -1 there, and what is left of S would carry its
// rounding: 2e-5 of it at g = -8, all of it at -18).
constexpr float kWeakG = -0.6931472f;
struct Decay {
    float by;
    bool weak;
};
__device__ __forceinline__ Decay decay_of(float g) {
    const bool weak = g >= kWeakG;  // (NaN: no)
    return {weak ? expm1f(g) : expf(g), weak};
}
__device__ __forceinline__ float decayed(Decay d, float x) { return fmaf(d.by, x, d.weak ? x : 0.0f); }

// Cumulative log decays are kept as the unevaluated sum of two floats (Knuth's
// two-sum): e^{c_i - c_j} of neighbouring tokens then stays exact to f32
// rounding however far c has fallen since the chunk's start (a reset in the
// chunk takes it to -128 and below).
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_add(Two a, Two b) {
    const float s = a.h + b.h;
    const float t = s - a.h;
    const float e = (a.h - (s - t)) + (b.h - t);
    const float l = a.l + b.l + e;
    Two r;
    r.h = s + l;
    r.l = l - (r.h - s);
    return r;
}
__device__ __forceinline__ float two_diff(Two a, Two b) { return (a.h - b.h) + (a.l - b.l); }

// One warp: inclusive sums of T = 32 * E values, lane i holding values
// i * E .. i * E + E - 1.
template <int E> __device__ __forceinline__ void warp_cumsum(const float (&x)[E], Two (&c)[E]) {
    const int lane = threadIdx.x & 31;
    c[0] = {x[0], 0.0f};
#pragma unroll
    for (int e = 1; e < E; e++) c[e] = two_add(c[e - 1], {x[e], 0.0f});
    Two run = c[E - 1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two up = {__shfl_up_sync(kFull, run.h, o), __shfl_up_sync(kFull, run.l, o)};
        if (lane >= o) run = two_add(up, run);
    }
    const Two before = {__shfl_up_sync(kFull, run.h, 1), __shfl_up_sync(kFull, run.l, 1)};
    if (lane > 0) {
#pragma unroll
        for (int e = 0; e < E; e++) c[e] = two_add(before, c[e]);
    }
}

}  // namespace la
}  // namespace ss
