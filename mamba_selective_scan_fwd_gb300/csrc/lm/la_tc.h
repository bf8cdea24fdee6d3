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
    CUtensorMap q, k, v, dy, y;
};

// How a walk over units (direction, batch row, head, 64 value channels; in this
// order, the last fastest) is cut: the first `whole` units are one block each, the other
// `cut` units K segments of seg tokens.  A cut unit's segments but the last are
// walked twice: a sum pass gives the state each segment starts from.
struct TcPlan {
    int64_t whole, cut, K, seg;
    int64_t blocks() const { return whole + cut * K; }
};

// slots: blocks that run at once (two on an SM in the forward, one in the
// state walk).  Full rounds of whole units, and the last partial round cut so
// that it fills the SMs, where that costs less than running it uncut.  Costs in
// chunks' time: a round of blocks, half as much for the sum pass, 3 for the two
// launches that cutting adds.  (bf16, cut against uncut: 4 x 4096 tokens x 80 heads 204
// and 283 us, 4096 x 24 heads 47 and 125, 131072 x 16 heads 349 and 3323; backward of
// 2 x 4096 x 80 heads 401 and 414.)
inline TcPlan tc_plan(int64_t units, int64_t L, int64_t slots) {
    const int64_t chunks = ceil_div(L, kChunkTc), rest = units % slots;
    TcPlan best = {units, 0, 1, chunks * kChunkTc};
    if (rest == 0) return best;
    double least = (double)chunks;
    for (int64_t K = 2; K <= 256 && K <= chunks; K++) {
        const int64_t per = ceil_div(chunks, K);
        if (ceil_div(chunks, per) != K) continue;
        const double cost = (double)(ceil_div(rest * K, slots) * per) + 0.5 * (ceil_div(rest * (K - 1), slots) * per) + 3;
        if (cost < least) {
            least = cost;
            best = {units - rest, rest, K, per * kChunkTc};
        }
    }
    return best;
}

// An image of a state (N x 64, f32) for the backward: operand tiles of 64 * nb
// rows whose sum it is to 22 bits (f16: 2 parts of 11), 24 (bf16, N <= 64: 3 parts
// of 8) or 16 (bf16, N > 64: a third part finds no room in shared memory, and dg is
// good to 1e-6 instead of 4e-7).
template <bool F16, int NB> constexpr int kImageParts = !F16 && NB == 1 ? 3 : 2;
inline int64_t image_bytes(bool f16, int64_t N) {
    const int parts = N > 64 ? (f16 ? kImageParts<true, 2> : kImageParts<false, 2>)
                             : (f16 ? kImageParts<true, 1> : kImageParts<false, 1>);
    return (int64_t)parts * (N > 64 ? 2 : 1) * 8192;
}

// What a walk starts from and leaves, one for each direction.
struct TcDir {
    const float* init;   // state before its first token, or null
    float* last;         // state after its last token, or null
    void* images;        // [Bsz, H, ptiles, chunks] images of the state before each chunk
    float* image_scale;  // f16: the power of two each image was multiplied by (infinite: the state is zero)
};

// A walk in one direction (dirs = 1: forward), or the backward's two at once:
// units 0 .. and, from the middle of all units on, their reverse.
struct TcWalkArgs {
    TcMaps maps;
    Args a;
    TcPlan plan;
    TcDir dir[2];
    int dirs;
    float* seg_state;  // [cut, K, N, 64]: end states of the segments, then (after the carry) their start states
    float* seg_decay;  // [cut, K]
    int64_t chunks;
    int* status;
};

// The backward runs one block per SM.  bf16: the heads of all (batch row, chunk,
// group) in a row, in equal runs: dq and dk of a group that one block holds whole are
// outputs of that block, of one that is cut they are f32 parts (at most two a block:
// of the group its run begins in and of the one it ends in) that a second kernel
// adds up.
inline int64_t tc_bwd_blocks(int64_t heads) { return heads < kSms ? heads : kSms; }

// dq, dk: the outputs; parts: f32, in boxes of 32 columns (bf16: [2 blocks, 128, N];
// f16: [splits, Bsz, L, G, N], with splits > 1)
struct TcBwdMaps {
    CUtensorMap q, k, v, dy, dq, dk, dv, dq_part, dk_part;
};

struct TcBwdArgs {
    TcBwdMaps maps;
    Args a;
    const void *before, *after;               // images of H and R (as TcWalkArgs::images)
    const float *before_scale, *after_scale;  // f16: their scales
    int64_t chunks;
    float* dg;                 // [Bsz, L, H]; f16: [value tiles, Bsz, L, H]
    int splits;  // f16: parts of a group's dq and dk, one per head and value tile; bf16: 1
    void *dq, *dk;
    const float *dq_part, *dk_part;
    int* status;
};
cudaError_t launch_tc_bwd(const TcBwdArgs& w, cudaStream_t st);

cudaError_t launch_tc_fwd(const TcWalkArgs& w, cudaStream_t st);
cudaError_t launch_tc_state(const TcWalkArgs& w, bool sum, cudaStream_t st);
cudaError_t launch_tc_carry(const TcWalkArgs& w, cudaStream_t st);
cudaError_t launch_late_timeout(int* status, uint64_t limit_ns, cudaStream_t st);  // a wait that runs out, reported

}  // namespace la

// Library-wide state kept by api.cu: the current device's status word, and the
// driver's tensor-map encoder (null where it is missing, or while
// ss_set_copies_only keeps the library off TMA).
int device_status_word(int** out);
void* tensor_map_encoder();

}  // namespace ss
