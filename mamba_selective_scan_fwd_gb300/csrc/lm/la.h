// Head-decay linear attention: arguments, launch plans and workspace layouts
// shared by the C ABI (la_api.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../common.cuh"

namespace ss {
namespace la {

// Lets a kernel take `bytes` of dynamic shared memory; asked of the driver once
// per kernel and device.
template <auto Kernel> cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// An input of [Bsz, L, heads, width]: the last two dimensions contiguous, the
// first two with strides in elements.
struct In {
    const void* p;
    int64_t token, batch;
};

struct Args {
    In q, k, v, dy;          // dy: backward only
    const float* g;          // [Bsz, L, H], or [H] when g_per_head
    const float* h0;         // forward initial state, or null
    const float* dlast;      // gradient of the last state, or null (backward)
    const int32_t* lengths;  // [Bsz] or null
    int64_t Bsz, L, H, G, N, P;
    float scale;
    int dtype, g_per_head;
};

constexpr int kSms = 152;
constexpr int kMaxN = 128;

// ---------------------------------------------------------------- FP32 path
constexpr int kWalkP = 64;    // value channels per block of the token walk
constexpr int kWalkT = 16;    // tokens staged at a time (at most)
constexpr int kChunk32 = 64;  // tokens per chunk of the FP32 backward

// The token walk: every unit (direction, batch row, head, tile of value
// channels) is cut into K segments of seg tokens (the backward's are one chunk
// each: their start states are what it reads).
struct WalkPlan {
    int64_t K, seg;
};
// The K with the fewest tokens an SM walks: its blocks share it (fewer than the two or
// three that fit take as long as those), and a block's start and end are as long as 32
// tokens.  Cutting costs a sum pass (0.4 of a walk), two launches (as long as 160
// tokens) and the traffic of the segments' states (a token for 12 of them).
inline WalkPlan walk_plan(int64_t units, int64_t L, int64_t N) {
    const int64_t tiles = ceil_div(L, kWalkT);
    const int64_t fit = N > 64 ? 2 : 3;
    auto load = [&](int64_t blocks) { const int64_t n = ceil_div(blocks, kSms); return n < fit ? fit : n; };
    WalkPlan best = {1, tiles * kWalkT};
    double least = (double)load(units) * (L + 32);
    for (int64_t K = 2; K <= 512 && K <= tiles; K += K < 64 ? 1 : 16) {
        const int64_t per = ceil_div(tiles, K);
        if (ceil_div(tiles, per) != K) continue;
        const double cost = (load(units * K) + 0.4 * load(units * (K - 1))) * (double)(per * kWalkT + 32) + 160 + units * K / 12;
        if (cost < 0.95 * least) {
            least = cost;
            best = {K, per * kWalkT};
        }
    }
    return best;
}

// What a walk starts from and leaves, one for each direction.
struct WalkDir {
    const float* init;   // state before the walk's first token, or null
    float* last;         // state after its last token, or null
};

// dirs = 1: the forward, whose sum pass leaves out the segment walked last; 2: the
// backward's states in both directions, from sums of all segments.
struct WalkArgs {
    Args a;
    WalkPlan plan;
    WalkDir dir[2];
    int dirs;
    float* seg_state;  // [dirs, Bsz, H, K, N, P]: end states of the segments, then (after the carry) their start states
    float* seg_decay;  // [dirs, Bsz, H, K]
    void* y;
    bool vec;          // runs of four values are whole and aligned
};

struct BwdArgs {
    Args a;
    const float* before;  // [Bsz, H, chunks, N, P] state before each chunk
    const float* after;   // [Bsz, H, chunks, N, P] adjoint of the state after each chunk
    int64_t chunks;
    void *dq, *dk, *dv;
    float* dg;            // [Bsz, L, H]
    float *dq_part, *dk_part;  // [splits, Bsz, L, G, N] f32 when splits > 1
    int splits;           // parts the heads of one group are divided into
};

cudaError_t launch_walk32(const WalkArgs& w, bool sum, cudaStream_t st);  // sum: the segments' end states; else y
cudaError_t launch_carry32(const WalkArgs& w, cudaStream_t st);
cudaError_t launch_bwd32(const BwdArgs& b, cudaStream_t st);
// out[i] = sum of the splits' part[., i] (n each), of one pair of arrays or (out2 given) of two
cudaError_t launch_sum_parts(const float* part, void* out, const float* part2, void* out2, int splits, int64_t n, int dtype,
                             cudaStream_t st);
// dg [rows, H] summed over rows into out [H]; part holds kDgParts * H floats
constexpr int kDgParts = 64;
cudaError_t launch_sum_rows(const float* dg, float* part, float* out, int64_t rows, int64_t H, cudaStream_t st);

struct StepArgs {
    const void *q, *k, *v;
    const float* g;
    float* state;
    const int32_t* slots;
    void* y;
    int64_t q_batch, k_batch, v_batch;
    int64_t Bsz, H, G, N, P, pool;
    float scale;
    int dtype, g_per_head;
};
cudaError_t launch_step(const StepArgs& s, cudaStream_t st);

}  // namespace la

struct GnormArgs {
    const void *x, *z, *dout;
    const float *weight, *bias;
    void *out, *dx, *dz;
    float *dweight, *dbias;
    float* part;  // backward: [blocks, 2, C] partial sums
    int64_t M, C, groups;
    float eps;
    int flags, dtype;
};
cudaError_t launch_gnorm_fwd(const GnormArgs& a, cudaStream_t st);
cudaError_t launch_gnorm_bwd(const GnormArgs& a, cudaStream_t st);
int64_t gnorm_bwd_blocks(int64_t M, int64_t C, int64_t groups);

}  // namespace ss
