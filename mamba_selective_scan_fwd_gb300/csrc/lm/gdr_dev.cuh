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

// One warp, lane = tokens 2 lane and 2 lane + 1 of a chunk: its cumulative log2 decays c, tail = e^{c_e - c_t} with e
// the end of the token's run of 16, and whether no run leaves 2^-64 .. 2^64 (then e^{c_i - c_j} inside one may be
// taken as e^{c_i - c_e} e^{c_e - c_j}).  Returns this lane's c.
struct Pair {
    la::Two c[2];
};
__device__ __forceinline__ Pair chunk_decays(const Args& a, int64_t b, int64_t t0, int64_t h, int nv, la::Two* c, float* tail, bool& flat) {
    const int lane = threadIdx.x & 31;
    float x[2];
#pragma unroll
    for (int i = 0; i < 2; i++) x[i] = 2 * lane + i < nv ? log_decay(a, b, t0 + 2 * lane + i, h) * la::kLog2e : 0.0f;
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

}  // namespace gdr
}  // namespace ss
