// Device helpers of the gated delta rule's kernels.
#pragma once

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

}  // namespace gdr
}  // namespace ss
