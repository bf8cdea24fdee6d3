// Device helpers of the gated delta rule's kernels.
#pragma once

#include "../simd.cuh"
#include "gdr.h"
#include "la_dev.cuh"

namespace ss {
namespace gdr {

using la::ldf;

__device__ __forceinline__ int64_t row_length(const Args& a, int64_t b) {
    if (!a.lengths) return a.L;
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : (n > a.L ? a.L : n);
}
__device__ __forceinline__ float log_decay(const Args& a, int64_t b, int64_t t, int64_t h) {
    return a.g ? la::clamp_g(a.g[(b * a.L + t) * a.H + h]) : 0.0f;
}

// Growth.  Where log decays are positive, tokens' values grow like 2^{C_t - m_t}, C the chunk's cumulative log2 decays and m the least
// of them so far (and of zero, the start), and so do the factors 2^{C_i - C_j} of later rows and earlier columns: one scale
// would not hold a tile of them.  So a token's values stand in units of 2^{d_t}, d_t = C_t - m_t rounded: with v / 2^d for v and y / 2^d for
// y the chunk's formulas are those of the decays c = C - d, whose differences 2^{c_i - c_j} = 2^{m_i - m_j}, nearly, are at most two.
// Adjoints grow the other way, like 2^{M_t - C_t}, M the largest from t on, and stand in units of that.  The products that take
// both meet in 2^{rise_t}, rise = M_t - m_t rounded.  Powers of two change no digit, and without growth d and rise are zero.
constexpr int kMostGrowth = 120;
__device__ __forceinline__ float power2(int d) { return __uint_as_float((uint32_t)(127 + d) << 23); }  // |d| <= 126

// One warp, lane = tokens 2 lane and 2 lane + 1 of a chunk, x: their log2 decays; the chunk's cumulative log2 decays c (less
// growth), tail = e^{c_e - c_t} with e the end of the token's run of 16, and whether no run leaves 2^-64 .. 2^64 (then e^{c_i - c_j}
// inside one may be taken as e^{c_i - c_e} e^{c_e - c_j}).  Returns this lane's c, d and rise, and what the decays add up to.
struct Pair {
    la::Two c[2], sum;
    int grow[2], rise[2];
};
__device__ __forceinline__ Pair chunk_decays(const float (&x)[2], la::Two* c, float* tail, bool& flat) {
    const int lane = threadIdx.x & 31;
    Pair p;
    la::warp_cumsum<2>(x, p.c);
    p.sum = p.c[1];
    p.grow[0] = p.grow[1] = p.rise[0] = p.rise[1] = 0;
    if (__any_sync(kFull, x[0] > 0.0f || x[1] > 0.0f)) {
        float least = fminf(0.0f, fminf(p.c[0].h, p.c[1].h)), most = fmaxf(p.c[0].h, p.c[1].h);  // of all tokens up to, and from this lane's
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float up = __shfl_up_sync(kFull, least, o), down = __shfl_down_sync(kFull, most, o);
            if (lane >= o) least = fminf(least, up);
            if (lane + o < 32) most = fmaxf(most, down);
        }
        float m = __shfl_up_sync(kFull, least, 1), M = __shfl_down_sync(kFull, most, 1);
        if (lane == 0) m = 0.0f;
        if (lane == 31) M = p.c[1].h;
        M = fmaxf(M, p.c[1].h);
        auto rounded = [](float x) { return fminf(fmaxf(rintf(x), 0.0f), (float)kMostGrowth); };
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float c = p.c[i].h;
            m = fminf(m, c);
            const float d = rounded(c - m);
            p.grow[i] = (int)d;
            p.rise[i] = (int)fminf(d + rounded((i ? M : fmaxf(M, c)) - c), (float)kMostGrowth);
            p.c[i] = la::two_add(p.c[i], {-d, 0.0f});
        }
    }
    const la::Two end = {__shfl_sync(kFull, p.c[1].h, lane | 7), __shfl_sync(kFull, p.c[1].l, lane | 7)};
    flat = true;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        c[2 * lane + i] = p.c[i];
        const float rel = la::two_diff(end, p.c[i]);
        flat = flat && fabsf(rel) <= 64.0f;  // (NaN: no)
        tail[2 * lane + i] = ex2a(rel);
    }
    flat = __all_sync(kFull, flat);
    return p;
}

// x[j] *= f e^{c_i - c_{j0 + j}} for columns up to `last`, 0 beyond: by runs of 16 with one exponential each where `flat` allows it
// (a factor beyond `last` may overflow: it is not used), else an exponential each.
template <int N>
__device__ __forceinline__ void pair_factors(float (&x)[N], const la::Two* c, const float* tail, bool flat, int j0, la::Two ci, float f, int last) {
    if (flat) {
#pragma unroll
        for (int r = 0; r < N; r += 16) {
            const float2 by = splat2(f * ex2a(la::two_diff(ci, c[j0 + r + 15])));
#pragma unroll
            for (int j = r; j < r + 16; j += 4) {
                const float4 t = *reinterpret_cast<const float4*>(tail + j0 + j);
                const float2 u = mul2(make_float2(x[j], x[j + 1]), mul2(by, make_float2(t.x, t.y)));
                const float2 v = mul2(make_float2(x[j + 2], x[j + 3]), mul2(by, make_float2(t.z, t.w)));
                x[j] = j0 + j <= last ? u.x : 0.0f;
                x[j + 1] = j0 + j + 1 <= last ? u.y : 0.0f;
                x[j + 2] = j0 + j + 2 <= last ? v.x : 0.0f;
                x[j + 3] = j0 + j + 3 <= last ? v.y : 0.0f;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j++) {
            const float e = f * ex2a(la::two_diff(ci, c[j0 + j])) * x[j];
            x[j] = j0 + j <= last ? e : 0.0f;
        }
    }
}

}  // namespace gdr
}  // namespace ss
