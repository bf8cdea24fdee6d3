/*
 * ss_gdr.h -- C ABI of the GB300 (sm_103a) gated delta rule and of the norm
 * with rotation that a layer puts on its queries and keys.  It extends ss.h and
 * ss_la.h (same library, same conventions: caller-owned device memory, nothing
 * allocated, no synchronisation, work enqueued on `stream`, checks before the
 * first launch, deterministic results).
 *
 * Gated delta rule, per batch row b and head h, with a state S of N x P:
 *
 *   u_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t)
 *   S_t = e^{g_t} S_{t-1} + k_t u_t^T             (S starts at h0, or at zero)
 *   y_t = scale * q_t S_t
 *
 * the recurrence S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T:
 * where linear attention (ss_la.h) only adds k v^T, each token first takes back
 * what the state already answers to its key.  It contracts while beta |k|^2 <= 2;
 * nothing here normalises q or k (ss_qknorm_fwd does).
 *
 * Layouts, as in ss_la.h.  q, k: io [Bsz, L, G, N], v, y, dy, dv: io [Bsz, L, H, P];
 * R = H / G heads of v share one head of q and k.  g (log decay, or NULL: no
 * gate), beta, dg, dbeta: f32 [Bsz, L, H].  States: f32 [Bsz, H, N, P].  lengths:
 * int32 [Bsz], the tokens of each row that count: later ones are not read as
 * numbers (they may hold NaN), give y = 0 and zero gradients and leave the state
 * alone.  q, k, v, dy may be slices of a wider projection: the last two dimensions
 * are contiguous, *_token / *_batch are distances in elements.  Outputs are
 * contiguous and overlap no input.
 *
 * exp(g) = 0 (g = -inf or below -128) resets the state.  g <= 0 is in range, and
 * so is positive g, which lets the state grow, as long as no run of tokens inside
 * 64 adds up to more than 60.  Any finite beta is in range on f32 inputs, and on
 * 16-bit ones as long as rates with beta |k|^2 > 2 do not multiply the state by more
 * than 2^16 inside 64 tokens.  Tokens of 64 share matrix products: a non-finite q,
 * k, v, g or beta may reach any y of its 64 tokens, and all later ones.
 *
 * Precision.  f32 inputs: as f32 sums have it.  16-bit inputs: every value that the
 * chunks of 64 tokens make has 22 bits, 16-bit outputs are rounded once, f32 ones
 * are good to 1e-6 of their norm.  A channel's values in a chunk (v's and the
 * state's share, and the adjoints) have 22 bits down to 2^-16 of the largest of
 * them and lose one a power of two below: what is left of a state, or of an adjoint,
 * that 64 tokens take below that is good by what it was, not by itself.  q and k of
 * bf16 are exact down to 2^-27 of the largest in their 64 tokens and head.
 *
 * io is f32, f16 or bf16 (`dtype`, as in ss.h); states, decays, rates, sums, dg,
 * dbeta and dh0 are f32, dq, dk and dv have the io type.  Any 1 <= N <= 128 and
 * P >= 1, any strides.  Inputs of q's, k's, v's and dy's kind, g, beta, lengths and
 * slots may start at any element; states, outputs and workspaces (h0, last_state,
 * dlast_state, state, y, dq, dk, dv, dg, dbeta, dh0) start on 16 bytes, else
 * SS_ERR_UNSUPPORTED: a view such as pool[i:i+1] does where H * N * P is a multiple
 * of four.
 */
#ifndef SS_GDR_H
#define SS_GDR_H

#include "ss.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    const void *q, *k, *v;
    const float *g;           /* or NULL: no decay */
    const float *beta;
    const float *h0;          /* or NULL: zero */
    const int32_t *lengths;   /* or NULL: every row has L tokens */
    void *y;
    float *last_state;        /* or NULL */
    void *workspace;          /* >= ss_gdr_fwd_workspace_bytes(...), 16-byte aligned */
    size_t workspace_bytes;
    int64_t q_token, q_batch, k_token, k_batch, v_token, v_batch;
    int64_t Bsz, L, H, G, N, P;
    float scale;
    int32_t dtype;
} ss_gdr_fwd_desc;

/* Bytes of device workspace; a pure function of its arguments. */
size_t ss_gdr_fwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype);

/* Forward.  With L = 0 last_state receives a copy of h0 (zeros without it). */
int ss_gdr_fwd(const ss_gdr_fwd_desc *desc, void *stream);

/*
 * Backward of sum(dy * y) + sum(dlast_state * last_state).  It recomputes the
 * states it needs from the forward's inputs.  dq and dk are summed over the heads
 * that share them.  dg is given exactly when g is, dh0 exactly when h0 is (else
 * SS_ERR_INVALID_PROBLEM).  With L = 0 dh0 receives a copy of dlast_state.
 */
typedef struct {
    const void *q, *k, *v;
    const float *g, *beta;
    const float *h0;
    const int32_t *lengths;
    const void *dy;
    const float *dlast_state; /* or NULL: zero */
    void *dq, *dk, *dv;
    float *dg;                /* iff g */
    float *dbeta;
    float *dh0;               /* iff h0 */
    void *workspace;          /* >= ss_gdr_bwd_workspace_bytes(...), 16-byte aligned */
    size_t workspace_bytes;
    int64_t q_token, q_batch, k_token, k_batch, v_token, v_batch, dy_token, dy_batch;
    int64_t Bsz, L, H, G, N, P;
    float scale;
    int32_t dtype;
} ss_gdr_bwd_desc;

size_t ss_gdr_bwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype);
int ss_gdr_bwd(const ss_gdr_bwd_desc *desc, void *stream);

/*
 * One token for each of Bsz sequences, in place on their states (the recurrence
 * above with S = state[slot]).  q, k io [Bsz, G, N], v, y io [Bsz, H, P], g (or
 * NULL) and beta f32 [Bsz, H]; state f32 [pool, H, N, P].  slots (int32 [Bsz], or
 * NULL: row b uses state b) names each row's state; a row whose slot lies outside
 * 0..pool-1 (-1 marks a padding row) gives y = 0 and touches no state.  Two rows of
 * one call must not name the same slot.  One kernel, no workspace.
 */
typedef struct {
    const void *q, *k, *v;
    const float *g, *beta;
    float *state;
    const int32_t *slots;
    void *y;
    int64_t q_batch, k_batch, v_batch;
    int64_t Bsz, H, G, N, P, pool;
    float scale;
    int32_t dtype;
} ss_gdr_step_desc;
int ss_gdr_step(const ss_gdr_step_desc *desc, void *stream);

/*
 * Norm of each head's channels of q and k, and the rotation by position, in one
 * pass.  Per token and head, over the N channels of x:
 *   n = x / sqrt(mean(x^2) + eps) * weight      (weight f32 [N] or NULL: 1)
 *   n = x / sqrt(sum(x^2) + eps) * weight       with SS_QKNORM_L2
 * then the first 2 * pairs channels are turned: channels i and i + pairs (or 2 i and
 * 2 i + 1 with SS_QKNORM_INTERLEAVED), i < pairs, by the angle position * freqs[i]:
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * freqs f32 [pairs] (radians a token; NULL with pairs = 0: no rotation), positions
 * int32 [Bsz, L], or NULL: token t of each row stands at t.  The product of position
 * and frequency is reduced to a fraction of a turn in integers: the angle is good to
 * 2^-26 turns and 2^-52 of the turns made, 2^-23 a radian a token and 2^31 tokens on.
 *
 * q io [Bsz, L, Hq, N], k io [Bsz, L, Hk, N], slices of a wider projection allowed;
 * the outputs are contiguous, and may be the inputs themselves where those are.
 * 1 <= N <= 256, 2 * pairs <= N.  All pointers but the workspace's may start at any
 * element.  Sums of squares are f32: the norm of a head is out of range above 1e19,
 * and below 1e-19 with eps = 0.
 */
enum { SS_QKNORM_L2 = 1, SS_QKNORM_INTERLEAVED = 2 };
typedef struct {
    const void *q, *k;
    const float *q_weight, *k_weight;
    const int32_t *positions;
    const float *freqs;
    void *q_out, *k_out;
    int64_t q_token, q_batch, k_token, k_batch;
    int64_t Bsz, L, Hq, Hk, N, pairs;
    float eps;
    int32_t flags, dtype, reserved; /* reserved: set to 0 */
} ss_qknorm_fwd_desc;
int ss_qknorm_fwd(const ss_qknorm_fwd_desc *desc, void *stream);

/*
 * Its gradient, from the forward's inputs and dq_out, dk_out (io, slices allowed):
 * dq, dk (io, contiguous) and dq_weight, dk_weight (f32 [N], exactly when their
 * weight is given), summed over batch, tokens and heads in a fixed order.
 */
typedef struct {
    const void *q, *k;
    const float *q_weight, *k_weight;
    const int32_t *positions;
    const float *freqs;
    const void *dq_out, *dk_out;
    void *dq, *dk;
    float *dq_weight, *dk_weight;
    void *workspace;          /* >= ss_qknorm_bwd_workspace_bytes(...), 16-byte aligned */
    size_t workspace_bytes;
    int64_t q_token, q_batch, k_token, k_batch, dq_token, dq_batch, dk_token, dk_batch; /* dq_, dk_: of dq_out, dk_out */
    int64_t Bsz, L, Hq, Hk, N, pairs;
    float eps;
    int32_t flags, dtype, reserved;
} ss_qknorm_bwd_desc;
size_t ss_qknorm_bwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t Hq, int64_t Hk, int64_t N, int dtype);
int ss_qknorm_bwd(const ss_qknorm_bwd_desc *desc, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_GDR_H */
