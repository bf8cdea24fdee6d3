// Fifth-generation tensor core helpers (inline PTX): tensor memory, matrix
// multiply descriptors, swizzled tiles, TMA copies of 4-D maps.
#pragma once

#include "../tma.cuh"
#include "la_dev.cuh"

namespace ss {
namespace la {

// ---------------------------------------------------------------- tensor memory
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {  // one whole warp
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {  // the same warp
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 or 32 columns of this warp's 32 lanes: thread = lane, x[i] = column i.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&x)[16]) {
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; i++) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&x)[32]) {
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; i++) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

// ---------------------------------------------------------------- matrix products
// Operand tiles live in shared memory as 128-byte rows of 64 16-bit values in
// the 128-byte swizzle (16-byte unit c of row r at c ^ (r & 7)), 1024-byte
// aligned: what a TMA box of 64 columns writes.  `kmajor`: the rows are the
// operand's M or N index (64 of the contraction along each row); otherwise
// the rows are the contraction index and `wide` is the distance between
// 64-column blocks of M or N.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t wide = 16) {
    return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)((wide >> 4) & 0x3fff) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
template <typename T> struct MmaType;
template <> struct MmaType<__half> { static constexpr uint32_t id = 0; };
template <> struct MmaType<__nv_bfloat16> { static constexpr uint32_t id = 1; };
// f32 accumulators; a_rows / b_rows: the operand's rows are the contraction index
template <typename T> __host__ __device__ constexpr uint32_t mma_desc(int m, int n, bool a_rows, bool b_rows) {
    return 1u << 4 | MmaType<T>::id << 7 | MmaType<T>::id << 10 | (a_rows ? 1u << 15 : 0u) | (b_rows ? 1u << 16 : 0u) |
           (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
        : "memory");
}
// The barrier completes when all matrix products issued so far by this thread have.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Waits of a block whose parts run on their own: the first wait that runs out
// sets *fail, and from then on no wait of the block waits, so that every part
// runs to its end at once.
__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t phase, volatile uint32_t* fail,
                                             uint64_t limit_ns = kWaitLimitNs) {
    if (*fail) return false;
    if (mbar_wait(bar, phase, limit_ns)) return true;
    *fail = 1;
    return false;
}

// The block's end, all its threads: a wait that ran out in any part (a part that ended
// before it cannot tell) is noted in the status word, what may still be in flight on
// the barriers `bars` of copies and products is waited for (one of a barrier's two
// phases is over already, the other gets kDrainLimitNs), and tensor memory is freed.
constexpr uint64_t kDrainLimitNs = 100000000ull;
template <int N>
__device__ __forceinline__ void end_block(volatile uint32_t* fail, int* status, uint64_t* const (&bars)[N], uint32_t tm, uint32_t cols) {
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x < 32) {
        if (*fail) {
            if (threadIdx.x == 0) {
                atomicOr(status, kDevWaitTimeout);
                for (int i = 0; i < N; i++) {
                    mbar_wait(bars[i], 0, kDrainLimitNs);
                    mbar_wait(bars[i], 1, kDrainLimitNs);
                }
            }
        }
        __syncwarp();
        tmem_free(tm, cols);
    }
}

// ---------------------------------------------------------------- copies
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}
// The same box, or `bytes` from p, into the L2 cache only, for a copy issued later
// (2 x 4096 tokens, 80 heads: the whole backward takes 401 us with it, 420 without).
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
__device__ __forceinline__ void bulk_prefetch(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_addr(src)), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ---------------------------------------------------------------- 16-bit pairs
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t x);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
    return {__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)};
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t x) {
    return __half22float2(*reinterpret_cast<__half2*>(&x));
}

template <typename T> constexpr bool kF16 = false;
template <> constexpr bool kF16<__half> = true;

// 16-byte unit c of row r of a swizzled tile
__device__ __forceinline__ uint4* unit(void* tile, int r, int c) {
    return reinterpret_cast<uint4*>(static_cast<char*>(tile) + r * 128 + ((c ^ (r & 7)) << 4));
}

// A power of two 2^e that takes `most` (>= 0) into [2^13, 2^14): f16 operands
// are scaled by it, so that neither their range nor their small values cost
// precision.  `most` bounds the operand as it will be, decays and weights in it:
// positive log decays make those larger than 1.  1 for 0, NaN and infinity.
__device__ __forceinline__ float f16_scale(float most) {
    const int e = (int)(__float_as_uint(most) >> 23) - 127;
    if (most == 0.0f || e >= 128) return 1.0f;
    int s = 13 - e;
    if (s > 126) s = 126;
    return __uint_as_float((uint32_t)(127 + s) << 23);
}

}  // namespace la
}  // namespace ss
