// Tensor-core path of the gated delta rule: arguments, plans and workspace layouts.
//
// A chunk is 64 tokens.  With c_i the cumulative log decay in it, cl its end, H the state
// before it, A_ij = beta_i e^{c_i - c_j} k_i . k_j (j < i) and M = (I + A)^{-1}:
//   U = M beta (V - e^c K H),   y = scale (e^c Q H + P U),   P_ij = e^{c_i - c_j} q_i . k_j (j <= i)
//   H <- e^{cl} H + (e^{cl - c} K)^T U
// (where decays grow, c and all values of a token less its growth: gdr_dev.cuh.)  M and P do not depend on the state: a first kernel makes them for all chunks at once
// (an "image" per chunk and head), a second walks the chunks.
#pragma once

#include "../tma.cuh"
#include "gdr.h"

namespace ss {
namespace gdr {

constexpr int kTileP = 128;  // value channels per block: the lanes of tensor memory
constexpr int kTileBytes = 8192;  // 64 rows of 64 16-bit values

// All operands that the kernels make are f16: two parts of one, scaled by a power of two, hold
// 22 bits (bf16's two hold 16).  So q and k become f16 once, scaled alike: every bf16 value
// within 2^27 of its tile's largest stays exact.  Tiles are 64 rows of 64 values in 128-byte rows,
// swizzled as TMA would.
//
// Keys: per (batch row, chunk, head of q and k), for each 64 columns a tile of K and one of Q,
// rows past the row's length zero.
constexpr int key_bytes(int64_t N) { return (N > 64 ? 4 : 2) * kTileBytes; }
// Image: per (batch row, head, chunk) tiles of M and of P, two parts each, then the chunk's factors.
struct ImageHead {
    float up[kChunk];    // e^{c_t}
    float down[kChunk];  // e^{cl - c_t}
    float beta[kChunk];     // beta_t / grow_t
    float beta_up[kChunk];  // beta_t e^{c_t}
    float tail[kChunk];     // e^{c_e - c_t}, e the end of the token's run of 16 (chunk_decays)
    float2 c[kChunk];       // c_t in units of log 2, the sum of two floats
    __nv_bfloat16 grow[kChunk];  // growth: a token's values are in units of this power of two, 2^{d_t}
    float by;            // the chunk's decay as la::Decay
    int32_t weak;
    float inv_k, inv_q, inv_m, inv_p;  // what undoes the scales of K, Q, M and P
    float most_k, most_q, most_m;  // largest values of K, Q and M
    int32_t flat;              // whether tail may stand for differences inside a run
    int32_t grown;             // whether any token's growth is not one
    int8_t rise[kChunk];       // log2 of the unit of values over that of adjoints
    float pad[5];
};
static_assert(sizeof(ImageHead) == 2048, "bulk copies are multiples of 16 bytes");
constexpr int kImageBytes = 4 * kTileBytes + (int)sizeof(ImageHead);
// The backward's images hold P in the adjoints' units.  Where a chunk grows, M and the factors in those units are in a place
// of their own beside the images, which only the walk of the adjoints reads.
constexpr int kTurnedBytes = 2 * kTileBytes + (int)sizeof(ImageHead);

struct PrepArgs {
    CUtensorMap q, k;  // {width, heads, L, Bsz}, boxes of 64 columns x 64 tokens
    Args a;
    int64_t chunks;
    int splits;        // blocks the heads of a group are divided into
    char* keys;        // [Bsz, chunks, G]
    char* images;      // [Bsz, H, chunks]
    char* turned;      // the same, of chunks that grow; null: forward
    int* status;
};
cudaError_t launch_prep(const PrepArgs& w, cudaStream_t st);

// f16 images as the walks hold them, transposed: pieces of 128 value channels p by 64, one scale each image.  The
// state (or its adjoint): [part][64 states n][p][64].  U and X: [part][p][64 tokens].  dY: [p][64 tokens], exact.
constexpr int kPieceBytes = 2 * kTileBytes;
__host__ __device__ constexpr int state_bytes(int nb) { return 2 * nb * kPieceBytes; }
constexpr int kRowsBytes = 2 * kPieceBytes;

// How the walks over time are cut: K segments of seg chunks.  All but the last are first walked
// for what they do to a state: from zero (E), and without v from the identity (Phi), so that
// S -> Phi S + E.
struct TcPlan {
    int64_t K, seg;
};

struct TcWalkArgs {
    CUtensorMap v, y;
    Args a;
    TcPlan plan;
    int64_t chunks;
    const char *keys, *images;
    const float* init;  // h0, or null (plan.K == 1)
    float* last;        // or null
    float* seg_state;   // [Bsz, H, K, N, P]: E of each segment, then (after the carry) the states they start from
    float* seg_phi;     // [Bsz, H, K, N, N], transposed
    float* seg_phi_t;   // the backward's: the same as it is
    void* yp;           // y again, for rows that no copy writes
    char *states, *us;  // kTcKeep: images [Bsz, H, value tiles, chunks]
    float *state_inv, *u_inv;  // what undoes each image's scale
    int* status;
};
// The backward's walk over the chunks from the last: x and, as images like the forward's, the state's
// adjoint after each chunk and X.
struct TcBackArgs {
    const char* turned;
    const char* dys;    // images of dY
    const float* dy_inv;
    const float* init;  // gradient of the last state, or null
    float* last;        // dh0, or null
    char *states, *xs;
    float *state_inv, *x_inv;
    float* seg_state;   // what a segment does to an adjoint of zero, then the adjoints they start from
};
cudaError_t launch_dy(const Args& a, int64_t chunks, const char* images, char* dys, float* dy_inv, cudaStream_t st);
// What is left of the backward, one chunk at a time.
struct TcChunkArgs {
    Args a;
    int64_t chunks;
    int splits;         // parts a group's heads are divided into
    const char *keys, *images, *before, *after, *us, *xs, *dys;
    const float *before_inv, *after_inv, *u_inv, *x_inv, *dy_inv;
    void *dq, *dk, *dv;
    float *dq_part, *dk_part;  // [splits, Bsz, L, G, N], with splits > 1
    float *dg, *dbeta;
    int* status;
};
// kTcY: y and the last state.  kTcSum: what each segment does to a state.  kTcKeep: for the backward, the
// state before each chunk and U, as operand images.
enum TcWalkMode { kTcY, kTcSum, kTcKeep };
cudaError_t launch_tc_walk(const TcWalkArgs& w, TcWalkMode mode, cudaStream_t st);
cudaError_t launch_tc_sums(const TcWalkArgs& w, const TcBackArgs& r, cudaStream_t st);  // the backward's, plan.K > 1
cudaError_t launch_tc_carry(const TcWalkArgs& w, const TcBackArgs* r, cudaStream_t st);
cudaError_t launch_tc_walks(const TcWalkArgs& w, const TcBackArgs& r, cudaStream_t st);  // kTcKeep and the backward's, at once
cudaError_t launch_tc_chunks(const TcChunkArgs& c, cudaStream_t st);

}  // namespace gdr

int device_status_word(int** out);
void* tensor_map_encoder();

}  // namespace ss
