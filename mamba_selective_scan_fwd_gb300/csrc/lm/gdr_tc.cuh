// What the delta rule's tensor-core kernels share.
#pragma once

#include "gdr_tc.h"
#include "tc.cuh"
#include "gdr_dev.cuh"

namespace ss {
namespace gdr {

// Products are issued by one warp as a whole, its operands the same in all lanes, by the one lane elected here.  (As fast as
// by one thread of a divergent warp: what a chain of products of 128 lanes and 16 terms waits for is the products
// themselves, 79 cycles each with 64 columns, 94 with 128, measured.)
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// The first try does not look whether another wait has run out.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t phase, volatile uint32_t* fail) {
    return mbar_try_wait(bar, phase) || la::wait_or_fail(bar, phase, fail);
}
// A whole warp's: all lanes get the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t phase, volatile uint32_t* fail) { return __all_sync(kFull, wait(bar, phase, fail)); }

}  // namespace gdr
}  // namespace ss
