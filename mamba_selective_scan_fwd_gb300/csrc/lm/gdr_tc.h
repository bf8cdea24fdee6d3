// Tensor-core path of the gated delta rule: arguments, plans and workspace layouts.
//
// A chunk is 64 tokens.  With c_i the cumulative log decay in it, cl its end, H the state
// before it, A_ij = beta_i e^{c_i - c_j} k_i . k_j (j < i) and M = (I + A)^{-1}:
//   U = M beta (V - e^c K H),   y = scale (e^c Q H + P U),   P_ij = e^{c_i - c_j} q_i . k_j (j <= i)
//   H <- e^{cl} H + (e^{cl - c} K)^T U
// M and P do not depend on the state: a first kernel makes them for all chunks at once
// (an "image" per chunk and head), a second walks the chunks.
#pragma once

#include "../tma.cuh"
#include "gdr.h"

namespace ss {
namespace gdr {

constexpr int kTileP = 128;  // value channels per block: the lanes of tensor memory
constexpr int kTileBytes = 8192;  // 64 rows of 64 16-bit values

// An image: tiles of 64 x 64 (128-byte rows, swizzled as TMA would): M in two bf16 parts,
// P in `parts` bf16 parts, then the chunk's factors.
struct ImageHead {
    float up[kChunk];    // e^{c_t}
    float down[kChunk];  // e^{cl - c_t}
    float beta[kChunk];
    float by;            // the chunk's decay as la::Decay
    int32_t weak;
    float pad[62];
};
static_assert(sizeof(ImageHead) == 1024, "bulk copies are multiples of 16 bytes");
__host__ __device__ constexpr int image_bytes(int parts) { return (2 + parts) * kTileBytes + (int)sizeof(ImageHead); }
// parts of P: y is good to the io type's half step with one in bf16, with two in f16
constexpr int fwd_parts(int dtype) { return dtype == 1 ? 2 : 1; }

struct PrepArgs {
    CUtensorMap q, k;  // {width, heads, L, Bsz}, boxes of 64 columns x 64 tokens
    Args a;
    int64_t chunks;
    int splits;        // blocks the heads of a group are divided into
    char* images;      // [Bsz, H, chunks]
    int* status;
};
cudaError_t launch_prep(const PrepArgs& w, int parts, cudaStream_t st);

// How the walks over time are cut: K segments of seg chunks.  All but the last are first walked
// for what they do to a state: from zero (E), and without v from the identity (Phi), so that
// S -> Phi S + E.
struct TcPlan {
    int64_t K, seg;
};

struct TcWalkArgs {
    CUtensorMap q, k, v, y;
    Args a;
    TcPlan plan;
    int64_t chunks;
    const char* images;
    const float* init;  // h0, or null (plan.K == 1)
    float* last;        // or null
    float* seg_state;   // [Bsz, H, K, N, P]: E of each segment, then (after the carry) the states they start from
    float* seg_phi;     // [Bsz, H, K, N, N]
    void* yp;           // y again, for rows that no copy writes
    int* status;
};
enum TcWalkMode { kTcY, kTcSum };
cudaError_t launch_tc_walk(const TcWalkArgs& w, TcWalkMode mode, cudaStream_t st);
cudaError_t launch_tc_carry(const TcWalkArgs& w, cudaStream_t st);

}  // namespace gdr

int device_status_word(int** out);
void* tensor_map_encoder();

}  // namespace ss
