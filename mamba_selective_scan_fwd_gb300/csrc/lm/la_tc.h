// Tensor-core path of the linear attention: arguments and plans.
#pragma once

#include "../tma.cuh"
#include "la.h"

namespace ss {
namespace la {

constexpr int kChunkTc = 128;  // tokens per chunk
constexpr int kTileP = 64;     // value channels per block

// 4-D maps {width, heads, L, Bsz}, boxes of 64 columns x 128 tokens.
struct TcMaps {
    CUtensorMap q, k, v, dy, y, dv;
};

// Segments of the tensor-core walk: two blocks run on an SM, so K is the
// number of segments with the least rounds of blocks times chunks per segment;
// cutting costs a second reading of k and v (the sum pass, about 0.6 of a walk)
// and two more launches (about two chunks' time).
inline WalkPlan tc_walk_plan(int64_t units, int64_t L) {
    const int64_t chunks = ceil_div(L, kChunkTc), slots = 2 * kSms;
    WalkPlan best = {1, chunks * kChunkTc};
    double least = (double)ceil_div(units, slots) * chunks;
    for (int64_t K = 2; K <= 256 && K <= chunks / 2; K++) {
        const int64_t per = ceil_div(chunks, K), segs = ceil_div(chunks, per);
        if (segs != K) continue;
        const double cost = (double)ceil_div(units * K, slots) * per + 0.6 * ceil_div(units * (K - 1), slots) * per + 2;
        if (cost < 0.95 * least) {
            least = cost;
            best = {K, per * kChunkTc};
        }
    }
    return best;
}

struct TcWalkArgs {
    TcMaps maps;
    Args a;
    WalkPlan plan;
    const float* init;
    float* seg_state;
    float* seg_decay;
    float* last;
    void* images;        // [Bsz, H, ptiles, chunks] of (high, low) operand tiles of the state before each chunk
    float* image_scale;  // f16: the power of two each image was multiplied by
    int64_t chunks;
    int* status;
};

cudaError_t launch_tc_fwd(const TcWalkArgs& w, cudaStream_t st);
cudaError_t launch_tc_state(const TcWalkArgs& w, bool reverse, bool sum, cudaStream_t st);

}  // namespace la

// Library-wide state kept by api.cu: the current device's status word, and the
// driver's tensor-map encoder (null where it is missing, or while
// ss_set_copies_only keeps the library off TMA).
int device_status_word(int** out);
void* tensor_map_encoder();

}  // namespace ss
