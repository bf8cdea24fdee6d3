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

// One warp, lane = tokens 2 lane and 2 lane + 1 of a chunk, x: their log2 decays; the chunk's cumulative log2 decays c, tail = e^{c_e - c_t} with e
// the end of the token's run of 16, and whether no run leaves 2^-64 .. 2^64 (then e^{c_i - c_j} inside one may be
// taken as e^{c_i - c_e} e^{c_e - c_j}).  Returns this lane's c.
struct Pair {
    la::Two c[2];
};
__device__ __forceinline__ Pair chunk_decays(const float (&x)[2], la::Two* c, float* tail, bool& flat) {
    const int lane = threadIdx.x & 31;
    Pair p;
    la::warp_cumsum<2>(x, p.c);
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
