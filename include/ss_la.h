/*
 * ss_la.h -- C ABI of the GB300 (sm_103a) linear attention with one decay per
 * head, and of the gated group norm that a layer puts on its output.  It
 * extends ss.h (same library, same conventions: caller-owned device memory,
 * nothing allocated, no synchronisation, work enqueued on `stream`, checks
 * before the first launch, deterministic results).
 *
 * Linear attention, per batch row b and head h, with a state S of N x P:
 *
 *   S_t = exp(g[b,t,h]) * S_{t-1} + k[b,t,h/R,:]^T v[b,t,h,:]     (S starts at h0, or at zero)
 *   y[b,t,h,:] = scale * q[b,t,h/R,:] S_t
 *
 * R = H / G heads of v share one head of q and k.  It is the recurrence of
 * ss.h with the decay of a channel's N states replaced by one scalar per
 * head, so that whole chunks of tokens become matrix products.
 *
 * Layouts.  q, k: io [Bsz, L, G, N].  v, y, dy, dv: io [Bsz, L, H, P].  g, dg:
 * f32 [Bsz, L, H], or [H] when g_per_head (one decay per head for all
 * tokens).  States (h0, last_state, dh0, dlast_state): f32 [Bsz, H, N, P].
 * lengths: int32 [Bsz].  Outputs are contiguous.  The inputs q, k, v, dy may
 * be slices of a wider projection: the last two dimensions are contiguous,
 * and *_token / *_batch give the distance in elements between tokens and
 * between batch rows.
 *
 * lengths cuts batch row b to its first lengths[b] tokens (values outside
 * 0..L are clamped): later tokens are not read as numbers (they may hold NaN),
 * give y = 0 and zero gradients whatever the row's own tokens hold, and leave the
 * state alone.
 *
 * g is a log decay.  exp(g) = 0 (g = -inf or below -128) resets the state.
 * Positive g lets it grow, in every type: the result is finite wherever it can be
 * represented, as long as no run of tokens inside 128 adds up to more than 60.
 * A chunk's scores are matrix products and its decays are taken from the ends of
 * runs of 32 tokens, so a non-finite q, k, v or g may reach any y of its chunk.
 *
 * Types.  io is f32, f16 or bf16 (`dtype`, as in ss.h).  States, decays, sums
 * and dg, dh0 are f32.  dq, dk, dv have the io type: they feed the
 * projections' 16-bit products, and 16-bit gradients halve what the backward
 * writes.
 *
 * Any 1 <= N <= 128 and P >= 1, any strides, any token-aligned pointers:
 * 16-bit inputs whose N, P, strides and pointers are multiples of 16 bytes
 * run on the tensor cores, everything else on the FP32 units.
 */
#ifndef SS_LA_H
#define SS_LA_H

#include "ss.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    const void *q, *k, *v;
    const float *g;
    const float *h0;          /* or NULL: zero */
    const int32_t *lengths;   /* or NULL: every row has L tokens */
    void *y;
    float *last_state;        /* or NULL */
    void *workspace;          /* >= ss_la_fwd_workspace_bytes(...), 16-byte aligned */
    size_t workspace_bytes;
    int64_t q_token, q_batch, k_token, k_batch, v_token, v_batch;
    int64_t Bsz, L, H, G, N, P;
    float scale;
    int32_t dtype, g_per_head, reserved; /* reserved: set to 0 */
} ss_la_fwd_desc;

/* Bytes of device workspace; a pure function of its arguments (the larger of what
 * the tensor cores' and the FP32 units' path need: strides and pointers, which
 * decide between them, are not known here). */
size_t ss_la_fwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype);

/* Forward.  With L = 0 last_state receives a copy of h0 (zeros without it). */
int ss_la_fwd(const ss_la_fwd_desc *desc, void *stream);

/*
 * Backward of sum(dy * y) + sum(dlast_state * last_state).  It recomputes the
 * states it needs from the forward's inputs.  dq and dk are summed over the
 * heads that share them, dg (g_per_head) over batch and tokens.  dh0 is given
 * exactly when h0 is (else SS_ERR_INVALID_PROBLEM).  With L = 0 dh0 receives
 * a copy of dlast_state (zeros without it), and a per-head dg zeros.
 */
typedef struct {
    const void *q, *k, *v;
    const float *g;
    const float *h0;
    const int32_t *lengths;
    const void *dy;
    const float *dlast_state; /* or NULL: zero */
    void *dq, *dk, *dv;
    float *dg;
    float *dh0;               /* iff h0 */
    void *workspace;          /* >= ss_la_bwd_workspace_bytes(...), 16-byte aligned */
    size_t workspace_bytes;
    int64_t q_token, q_batch, k_token, k_batch, v_token, v_batch, dy_token, dy_batch;
    int64_t Bsz, L, H, G, N, P;
    float scale;
    int32_t dtype, g_per_head, reserved;
} ss_la_bwd_desc;

size_t ss_la_bwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype);
int ss_la_bwd(const ss_la_bwd_desc *desc, void *stream);

/*
 * One token for each of Bsz sequences, in place on their states:
 *   state[slot] <- exp(g[b,h]) * state[slot] + k^T v;   y = scale * q state[slot]   (new state)
 * q, k io [Bsz, G, N], v, y io [Bsz, H, P], g f32 [Bsz, H] or [H]; state f32
 * [pool, H, N, P].  slots (int32 [Bsz], or NULL: row b uses state b) names
 * each row's state; a row whose slot lies outside 0..pool-1 (-1 marks a
 * padding row) gives y = 0 and touches no state.  Two rows of one call must
 * not name the same slot.  One kernel, no workspace.
 */
typedef struct {
    const void *q, *k, *v;
    const float *g;
    float *state;
    const int32_t *slots;
    void *y;
    int64_t q_batch, k_batch, v_batch;
    int64_t Bsz, H, G, N, P, pool;
    float scale;
    int32_t dtype, g_per_head, reserved;
} ss_la_step_desc;
int ss_la_step(const ss_la_step_desc *desc, void *stream);

/*
 * Runs one block on `stream` one part of which waits, for limit_ns nanoseconds
 * (0 .. 2e9; else SS_ERR_INVALID_PROBLEM), on a barrier nothing completes while
 * the others are over, and which ends as the tensor-core kernels above do: the
 * wait is reported in the status word that ss_device_status reads.  For testing
 * that path without any failure of the GPU.
 */
int ss_la_selftest_wait_timeout(int64_t limit_ns, void *stream);

/*
 * Group norm over groups of C / groups adjacent channels of each token (at most
 * 8192, else SS_ERR_UNSUPPORTED), with an activation:
 *   norm(a)  = (a - mean(a)) / sqrt(var(a) + eps) * weight + bias   per group; without SS_GNORM_CENTER
 *              a / sqrt(mean(a^2) + eps) * weight + bias
 *   z given, SS_GNORM_GATE_FIRST not set: out = norm(x) * silu(z)
 *   z given, SS_GNORM_GATE_FIRST set:     out = norm(x * silu(z))
 *   z NULL:                               out = silu(norm(x))
 * Statistics are taken inside each token, so that a causal model may use it.
 * x, z, out io [M, C] contiguous; weight, bias f32 [C], each may be NULL (1 and
 * 0).  The backward gives dx, dz (io; dz exactly when z is given) and dweight,
 * dbias (f32; exactly when weight, bias are), summed over tokens in a fixed
 * order.  M = 0 is valid: dweight and dbias are zero then.
 */
enum { SS_GNORM_CENTER = 1, SS_GNORM_GATE_FIRST = 2 };
int ss_gnorm_fwd(const void *x, const float *weight, const float *bias, const void *z, void *out, int64_t M, int64_t C,
                 int64_t groups, float eps, int flags, int dtype, void *stream);
size_t ss_gnorm_bwd_workspace_bytes(int64_t M, int64_t C, int64_t groups, int dtype);
int ss_gnorm_bwd(const void *x, const float *weight, const float *bias, const void *z, const void *dout, void *dx,
                 void *dz, float *dweight, float *dbias, int64_t M, int64_t C, int64_t groups, float eps, int flags,
                 int dtype, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_LA_H */
