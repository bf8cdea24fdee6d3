// C ABI of the gated delta rule and the q / k norm (include/ss_gdr.h).  Everything is
// checked before the first CUDA call; on error nothing is written.
#include "gdr.h"
#include "ss_gdr.h"

using namespace ss;
using namespace ss::gdr;

namespace {

bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool known(int dtype) { return dtype == SS_F32 || dtype == SS_F16 || dtype == SS_BF16; }

int check_sizes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype) {
    if (Bsz < 0 || L < 0 || H < 1 || G < 1 || N < 1 || P < 1 || H % G != 0) return SS_ERR_INVALID_PROBLEM;
    if (!known(dtype) || N > kMaxN) return SS_ERR_UNSUPPORTED;
    // products stay inside int64, grids inside 2^31 - 1 blocks
    if (Bsz > (1 << 20) || L > (1ll << 31) || H > (1 << 16) || P > (1 << 16)) return SS_ERR_UNSUPPORTED;
    if (Bsz * H * ceil_div(P, 16) > (1ll << 24) || Bsz * L > (1ll << 36)) return SS_ERR_UNSUPPORTED;
    if (Bsz * H * ceil_div(P, 16) * ceil_div(L, kChunk) >= (1ll << 31)) return SS_ERR_UNSUPPORTED;
    return SS_OK;
}

bool empty(int64_t Bsz, int64_t L) { return Bsz == 0 || L == 0; }
bool strides_ok(int64_t token, int64_t batch) { return token >= 0 && batch >= 0 && token <= (1ll << 40) && batch <= (1ll << 48); }

// A run of the workspace, in bytes from its start.
struct Layout {
    size_t total = 0;
    size_t take(size_t bytes) {
        const size_t at = total;
        total = align_up(total + bytes, 256);
        return at;
    }
};

// The FP32 backward's workspace.
struct Bwd32 {
    int64_t chunks;
    size_t miss, x, before, after, dq, dk;
};
Bwd32 bwd32_layout(Layout& l, int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P) {
    Bwd32 b;
    b.chunks = ceil_div(L, kChunk);
    const size_t rows = (size_t)Bsz * L * H * P * 4, states = (size_t)Bsz * H * b.chunks * N * P * 4;
    b.miss = l.take(rows);
    b.x = l.take(rows);
    b.before = l.take(states);
    b.after = l.take(states);
    const size_t part = H > G ? (size_t)(H / G) * Bsz * L * G * N * 4 : 0;
    b.dq = l.take(part);
    b.dk = l.take(part);
    return b;
}

// The state that no token changes: a copy of the incoming one, or zeros.
int pass_state(float* to, const float* from, int64_t Bsz, int64_t H, int64_t N, int64_t P, cudaStream_t st) {
    const size_t bytes = (size_t)Bsz * H * N * P * 4;
    if (!to || bytes == 0) return SS_OK;
    const cudaError_t e = from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(to, 0, bytes, st);
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

template <typename D> Args args_of(const D& d) {
    Args a = {};
    a.q = {d.q, d.q_token, d.q_batch};
    a.k = {d.k, d.k_token, d.k_batch};
    a.v = {d.v, d.v_token, d.v_batch};
    a.g = d.g;
    a.beta = d.beta;
    a.h0 = d.h0;
    a.lengths = d.lengths;
    a.Bsz = d.Bsz; a.L = d.L; a.H = d.H; a.G = d.G; a.N = d.N; a.P = d.P;
    a.scale = d.scale;
    a.dtype = d.dtype;
    return a;
}

int check_norm(int64_t Bsz, int64_t L, int64_t Hq, int64_t Hk, int64_t N, int64_t pairs, float eps, int flags, int dtype) {
    if (Bsz < 0 || L < 0 || Hq < 1 || Hk < 1 || N < 1 || pairs < 0 || 2 * pairs > N || !(eps >= 0.0f)) return SS_ERR_INVALID_PROBLEM;
    if (flags & ~(SS_QKNORM_L2 | SS_QKNORM_INTERLEAVED)) return SS_ERR_INVALID_PROBLEM;
    if (!known(dtype) || N > 256 || Hq > (1 << 16) || Hk > (1 << 16)) return SS_ERR_UNSUPPORTED;
    if (Bsz > (1 << 20) || L > (1ll << 31) || Bsz * L > (1ll << 36)) return SS_ERR_UNSUPPORTED;
    return SS_OK;
}
template <typename D> NormArgs norm_args(const D& d) {
    NormArgs a = {};
    a.side[0].x = {d.q, d.q_token, d.q_batch};
    a.side[1].x = {d.k, d.k_token, d.k_batch};
    a.side[0].weight = d.q_weight;
    a.side[1].weight = d.k_weight;
    a.side[0].heads = d.Hq;
    a.side[1].heads = d.Hk;
    a.positions = d.positions;
    a.freqs = d.freqs;
    a.Bsz = d.Bsz; a.L = d.L; a.N = d.N; a.pairs = d.pairs;
    a.eps = d.eps; a.flags = d.flags; a.dtype = d.dtype;
    return a;
}

}  // namespace

extern "C" {

size_t ss_gdr_fwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype) {
    if (check_sizes(Bsz, L, H, G, N, P, dtype) != SS_OK || empty(Bsz, L)) return 0;
    return 0;
}

int ss_gdr_fwd(const ss_gdr_fwd_desc* d, void* stream) {
    if (!d) return SS_ERR_INVALID_PROBLEM;
    const int rc = check_sizes(d->Bsz, d->L, d->H, d->G, d->N, d->P, d->dtype);
    if (rc != SS_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!strides_ok(d->q_token, d->q_batch) || !strides_ok(d->k_token, d->k_batch) || !strides_ok(d->v_token, d->v_batch))
        return SS_ERR_INVALID_PROBLEM;
    if (misaligned16(d->y) || misaligned16(d->h0) || misaligned16(d->last_state) || misaligned16(d->workspace))
        return SS_ERR_UNSUPPORTED;
    if (empty(d->Bsz, d->L)) return pass_state(d->last_state, d->h0, d->Bsz, d->H, d->N, d->P, st);
    if (!d->q || !d->k || !d->v || !d->beta || !d->y) return SS_ERR_INVALID_PROBLEM;
    const size_t need = ss_gdr_fwd_workspace_bytes(d->Bsz, d->L, d->H, d->G, d->N, d->P, d->dtype);
    if (d->workspace_bytes < need || (need > 0 && !d->workspace)) return SS_ERR_WORKSPACE_TOO_SMALL;
    const Args a = args_of(*d);
    WalkArgs w = {};
    w.a = a;
    w.init = a.h0;
    w.last = d->last_state;
    w.y = d->y;
    return launch_walk(w, kWalkY, st) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

size_t ss_gdr_bwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype) {
    if (check_sizes(Bsz, L, H, G, N, P, dtype) != SS_OK || empty(Bsz, L)) return 0;
    Layout l;
    bwd32_layout(l, Bsz, L, H, G, N, P);
    return l.total;
}

int ss_gdr_bwd(const ss_gdr_bwd_desc* d, void* stream) {
    if (!d) return SS_ERR_INVALID_PROBLEM;
    const int rc = check_sizes(d->Bsz, d->L, d->H, d->G, d->N, d->P, d->dtype);
    if (rc != SS_OK) return rc;
    if ((d->h0 == nullptr) != (d->dh0 == nullptr)) return SS_ERR_INVALID_PROBLEM;
    if (!strides_ok(d->q_token, d->q_batch) || !strides_ok(d->k_token, d->k_batch) ||
        !strides_ok(d->v_token, d->v_batch) || !strides_ok(d->dy_token, d->dy_batch))
        return SS_ERR_INVALID_PROBLEM;
    const void* ptrs[] = {d->h0, d->dlast_state, d->dq, d->dk, d->dv, d->dg, d->dbeta, d->dh0, d->workspace};
    for (const void* p : ptrs)
        if (misaligned16(p)) return SS_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (empty(d->Bsz, d->L)) return pass_state(d->dh0, d->dlast_state, d->Bsz, d->H, d->N, d->P, st);
    if ((d->g == nullptr) != (d->dg == nullptr)) return SS_ERR_INVALID_PROBLEM;
    if (!d->q || !d->k || !d->v || !d->beta || !d->dy || !d->dq || !d->dk || !d->dv || !d->dbeta) return SS_ERR_INVALID_PROBLEM;
    const size_t need = ss_gdr_bwd_workspace_bytes(d->Bsz, d->L, d->H, d->G, d->N, d->P, d->dtype);
    if (d->workspace_bytes < need || !d->workspace) return SS_ERR_WORKSPACE_TOO_SMALL;
    Args a = args_of(*d);
    a.dy = {d->dy, d->dy_token, d->dy_batch};
    a.dlast = d->dlast_state;
    char* ws = static_cast<char*>(d->workspace);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    Layout l;
    const Bwd32 bl = bwd32_layout(l, a.Bsz, a.L, a.H, a.G, a.N, a.P);
    WalkArgs w = {};
    w.a = a;
    w.chunks = bl.chunks;
    w.init = a.h0;
    w.rows = f32(bl.miss);
    w.states = f32(bl.before);
    if (launch_walk(w, kWalkKeep, st) != cudaSuccess) return SS_ERR_CUDA;
    w.init = a.dlast;
    w.last = d->dh0;
    w.y = d->dv;
    w.rows = f32(bl.x);
    w.states = f32(bl.after);
    if (launch_walk(w, kWalkBack, st) != cudaSuccess) return SS_ERR_CUDA;
    ChunkArgs c = {};
    c.a = a;
    c.miss = f32(bl.miss);
    c.x = f32(bl.x);
    c.before = f32(bl.before);
    c.after = f32(bl.after);
    c.chunks = bl.chunks;
    c.dq = d->dq;
    c.dk = d->dk;
    c.dq_part = f32(bl.dq);
    c.dk_part = f32(bl.dk);
    c.dg = d->dg;
    c.dbeta = d->dbeta;
    if (launch_chunks(c, st) != cudaSuccess) return SS_ERR_CUDA;
    if (a.H > a.G &&
        la::launch_sum_parts(c.dq_part, d->dq, c.dk_part, d->dk, (int)(a.H / a.G), a.Bsz * a.L * a.G * a.N, a.dtype, st) != cudaSuccess)
        return SS_ERR_CUDA;
    return SS_OK;
}

int ss_gdr_step(const ss_gdr_step_desc* d, void* stream) {
    if (!d) return SS_ERR_INVALID_PROBLEM;
    const int rc = check_sizes(d->Bsz, 1, d->H, d->G, d->N, d->P, d->dtype);
    if (rc != SS_OK) return rc;
    if (d->pool < 0 || (!d->slots && d->pool < d->Bsz) || d->q_batch < 0 || d->k_batch < 0 || d->v_batch < 0)
        return SS_ERR_INVALID_PROBLEM;
    if (misaligned16(d->state) || misaligned16(d->y)) return SS_ERR_UNSUPPORTED;
    if (d->Bsz == 0) return SS_OK;
    if (!d->q || !d->k || !d->v || !d->beta || !d->y || (!d->state && d->pool > 0)) return SS_ERR_INVALID_PROBLEM;
    const StepArgs s = {d->q, d->k, d->v, d->g, d->beta, d->state, d->slots, d->y, d->q_batch, d->k_batch, d->v_batch,
                        d->Bsz, d->H, d->G, d->N, d->P, d->pool, d->scale, d->dtype};
    return launch_step(s, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

int ss_qknorm_fwd(const ss_qknorm_fwd_desc* d, void* stream) {
    if (!d) return SS_ERR_INVALID_PROBLEM;
    const int rc = check_norm(d->Bsz, d->L, d->Hq, d->Hk, d->N, d->pairs, d->eps, d->flags, d->dtype);
    if (rc != SS_OK) return rc;
    if (!strides_ok(d->q_token, d->q_batch) || !strides_ok(d->k_token, d->k_batch)) return SS_ERR_INVALID_PROBLEM;
    if (empty(d->Bsz, d->L)) return SS_OK;
    if (!d->q || !d->k || !d->q_out || !d->k_out || (d->pairs > 0 && !d->freqs)) return SS_ERR_INVALID_PROBLEM;
    NormArgs a = norm_args(*d);
    a.side[0].out = d->q_out;
    a.side[1].out = d->k_out;
    return launch_qknorm(a, false, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

size_t ss_qknorm_bwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t Hq, int64_t Hk, int64_t N, int dtype) {
    if (check_norm(Bsz, L, Hq, Hk, N, 0, 0.0f, 0, dtype) != SS_OK || empty(Bsz, L)) return 0;
    return (size_t)(norm_blocks(Bsz * L, Hq, N) + norm_blocks(Bsz * L, Hk, N)) * N * 4;
}

int ss_qknorm_bwd(const ss_qknorm_bwd_desc* d, void* stream) {
    if (!d) return SS_ERR_INVALID_PROBLEM;
    const int rc = check_norm(d->Bsz, d->L, d->Hq, d->Hk, d->N, d->pairs, d->eps, d->flags, d->dtype);
    if (rc != SS_OK) return rc;
    if ((d->q_weight == nullptr) != (d->dq_weight == nullptr) || (d->k_weight == nullptr) != (d->dk_weight == nullptr))
        return SS_ERR_INVALID_PROBLEM;
    if (!strides_ok(d->q_token, d->q_batch) || !strides_ok(d->k_token, d->k_batch) || !strides_ok(d->dq_token, d->dq_batch) ||
        !strides_ok(d->dk_token, d->dk_batch))
        return SS_ERR_INVALID_PROBLEM;
    if (misaligned16(d->workspace)) return SS_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (empty(d->Bsz, d->L)) {
        for (float* w : {d->dq_weight, d->dk_weight})
            if (w && cudaMemsetAsync(w, 0, (size_t)d->N * 4, st) != cudaSuccess) return SS_ERR_CUDA;
        return SS_OK;
    }
    if (!d->q || !d->k || !d->dq_out || !d->dk_out || !d->dq || !d->dk || (d->pairs > 0 && !d->freqs)) return SS_ERR_INVALID_PROBLEM;
    if (!d->workspace || d->workspace_bytes < ss_qknorm_bwd_workspace_bytes(d->Bsz, d->L, d->Hq, d->Hk, d->N, d->dtype))
        return SS_ERR_WORKSPACE_TOO_SMALL;
    NormArgs a = norm_args(*d);
    a.side[0].d = {d->dq_out, d->dq_token, d->dq_batch};
    a.side[1].d = {d->dk_out, d->dk_token, d->dk_batch};
    a.side[0].out = d->dq;
    a.side[1].out = d->dk;
    a.side[0].dweight = d->dq_weight;
    a.side[1].dweight = d->dk_weight;
    a.part = static_cast<float*>(d->workspace);
    return launch_qknorm(a, true, st) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

}  // extern "C"
