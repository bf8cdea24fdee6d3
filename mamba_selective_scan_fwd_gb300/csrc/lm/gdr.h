// Gated delta rule and q / k norm: arguments, plans and launches shared by the C
// ABI (gdr_api.cu) and the kernels.
#pragma once

#include "la.h"

namespace ss {
namespace gdr {

using la::In;
using la::kMaxN;
using la::kSms;

struct Args {
    In q, k, v, dy;          // dy: backward only
    const float *g, *beta;   // [Bsz, L, H]; g may be null (no decay)
    const float* h0;         // initial state, or null
    const float* dlast;      // gradient of the last state, or null (backward)
    const int32_t* lengths;  // [Bsz] or null
    int64_t Bsz, L, H, G, N, P;
    float scale;
    int dtype;
};

constexpr int kChunk = 64;  // tokens whose pairs the backward forms (and the tensor cores' chunk)

// ---------------------------------------------------------------- FP32 path
constexpr int kWalkT = 16;  // tokens staged at a time
constexpr int kFour = 4;    // tokens whose products with the state are formed together
// lanes that share a value channel's N states, 16 each
inline int walk_lanes(int64_t N) { return N <= 16 ? 1 : N <= 32 ? 2 : N <= 64 ? 4 : 8; }

// What 16 tokens' products need that does not depend on the state, with c_t the log decay from the start of a
// token's four through it and cl its end.
struct Pairs {
    float kk[kWalkT][kFour], qk[kWalkT][kFour];  // e^{c_t - c_j} (k_t . k_j), (q_t . k_j), j of the token's four
    float up[kWalkT], down[kWalkT], beta[kWalkT];  // e^{c_t}, e^{cl - c_t}
    float by[kFour];                               // each four's decay as la::Decay
    int32_t weak[kFour];
    float pad[8];
};
static_assert(sizeof(Pairs) == 768, "whole 16-byte units");

// How the walks over time are cut: K segments of seg tiles, whole chunks.  They are first walked for what they do to a
// state: from zero (E), and without v from the identity (Phi), so that S -> Phi S + E, and for the adjoint from the end
// R -> Phi^T R + E'.
struct WalkPlan {
    int64_t K, seg;
};
WalkPlan walk_plan(int64_t heads, int64_t N, int64_t P, int64_t L, bool backward);

// kWalkSum: E or Phi; kWalkBackSum: E'
enum WalkMode { kWalkY, kWalkKeep, kWalkBack, kWalkSum, kWalkBackSum };
struct WalkArgs {
    Args a;
    const Pairs* pairs; // [Bsz, H, tiles of 16 tokens]
    const float* init;  // state (kWalkBack: adjoint) the walk starts from, or null
    float* last;        // where its last one goes, or null
    void* y;            // kWalkY: y; kWalkBack: dv
    float* rows;        // kWalkKeep: v - e^g S^T k (u / beta); kWalkBack: x; f32 [Bsz, L, H, P]
    float* states;      // kWalkKeep: before each chunk; kWalkBack: adjoint after it; f32 [Bsz, H, chunks, N, P]
    int64_t chunks;
    bool vec;           // f32, and runs of four values are whole and aligned: asynchronous copies
    WalkPlan plan;
    float* seg_state;   // f32 [Bsz, H, K, N, P], plan.K > 1: E (E'), then (after the carry) what each segment starts from
    float* seg_phi;     // f32 [Bsz, H, K, N, N]
};

struct ChunkArgs {
    Args a;
    const float *miss, *x;         // the walks' rows
    const float *before, *after;   // the walks' states
    int64_t chunks;
    void *dq, *dk;                 // io, when one head of v uses each head of q and k
    float *dq_part, *dk_part;      // else f32 [H / G, Bsz, L, G, N]
    float *dg, *dbeta;             // dg: may be null
};

cudaError_t launch_pairs(const Args& a, Pairs* pairs, cudaStream_t st);
cudaError_t launch_walk(const WalkArgs& w, cudaStream_t st);                          // kWalkY
cudaError_t launch_walks(const WalkArgs& keep, const WalkArgs& back, cudaStream_t st);  // the backward's two, at once
// What comes before them with plan.K > 1: the sums and the carry (back: of both directions).
cudaError_t launch_segments(const WalkArgs& w, const WalkArgs* back, cudaStream_t st);
cudaError_t launch_chunks(const ChunkArgs& c, cudaStream_t st);

struct StepArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    float* state;
    const int32_t* slots;
    void* y;
    int64_t q_batch, k_batch, v_batch;
    int64_t Bsz, H, G, N, P, pool;
    float scale;
    int dtype;
};
cudaError_t launch_step(const StepArgs& s, cudaStream_t st);

// ---------------------------------------------------------------- q / k norm
struct NormSide {  // q or k
    In x, d;                 // d: gradient of the output (backward)
    const float* weight;     // or null
    void* out;               // forward: the output; backward: the gradient of x
    float* dweight;          // backward, or null
    int64_t heads;
};
struct NormArgs {
    NormSide side[2];
    const int32_t* positions;
    const float* freqs;
    float* part;             // backward: [blocks of q, then of k][N] partial sums of the weights' gradients
    int64_t Bsz, L, N, pairs;
    float eps;
    int flags, dtype;
};
// Blocks of a side with `heads` heads beside `others` of the other: its part of what fits the SMs at once (a further
// block would wait for one of them to end), no more than there is work for (16 rows of 128 channels a block).  With
// kNormBlocks, the most that a launch takes, it sizes the workspace.
constexpr int kNormBlocks = 8;
int64_t norm_blocks(int64_t tokens, int64_t heads, int64_t others, int64_t N, int64_t per_sm);
cudaError_t launch_qknorm(const NormArgs& a, bool backward, cudaStream_t st);

}  // namespace gdr
}  // namespace ss
