// C ABI of the gated delta rule and the q / k norm (include/ss_gdr.h).  Everything is
// checked before the first CUDA call; on error nothing is written.
#include <cuda.h>

#include "gdr.h"
#include "gdr_tc.h"
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
    if (Bsz * H * ceil_div(P, 8) * ceil_div(L, kWalkT) >= (1ll << 31)) return SS_ERR_UNSUPPORTED;
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

size_t pairs_bytes(int64_t Bsz, int64_t L, int64_t H) { return (size_t)Bsz * H * ceil_div(L, kWalkT) * sizeof(Pairs); }

// The FP32 backward's workspace.
struct Bwd32 {
    int64_t chunks;
    WalkPlan plan;
    size_t pairs, miss, x, before, after, dq, dk, starts, ends, phi;
};
// The FP32 walks' segments, behind what else is there.
void segments(Layout& l, const WalkPlan& p, int64_t rows, int64_t N, int64_t P, size_t* starts, size_t* ends, size_t* phi) {
    const bool cut = p.K > 1;
    *starts = l.take(cut ? (size_t)rows * p.K * N * P * 4 : 0);
    if (ends) *ends = l.take(cut ? (size_t)rows * p.K * N * P * 4 : 0);
    *phi = l.take(cut ? (size_t)rows * p.K * N * N * 4 : 0);
}
struct Fwd32 {
    WalkPlan plan;
    size_t pairs, starts, phi;
};
Fwd32 fwd32_layout(Layout& l, int64_t Bsz, int64_t L, int64_t H, int64_t N, int64_t P) {
    Fwd32 f;
    f.plan = walk_plan(Bsz * H, N, P, L, false);
    f.pairs = l.take(pairs_bytes(Bsz, L, H));
    segments(l, f.plan, Bsz * H, N, P, &f.starts, nullptr, &f.phi);
    return f;
}
Bwd32 bwd32_layout(Layout& l, int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P) {
    Bwd32 b;
    b.chunks = ceil_div(L, kChunk);
    const size_t rows = (size_t)Bsz * L * H * P * 4, states = (size_t)Bsz * H * b.chunks * N * P * 4;
    b.pairs = l.take(pairs_bytes(Bsz, L, H));
    b.miss = l.take(rows);
    b.x = l.take(rows);
    b.before = l.take(states);
    b.after = l.take(states);
    const size_t part = H > G ? (size_t)(H / G) * Bsz * L * G * N * 4 : 0;
    b.dq = l.take(part);
    b.dk = l.take(part);
    b.plan = walk_plan(Bsz * H, N, P, L, true);
    segments(l, b.plan, Bsz * H, N, P, &b.starts, &b.ends, &b.phi);
    return b;
}

// ---------------------------------------------------------------- tensor-core path
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// [Bsz, L, heads, width] of 16-bit values as a map {width, heads, L, Bsz}, boxes of 64 columns
// by 64 tokens in the 128-byte swizzle; what lies outside reads as zero.
bool tc_map(EncodeTiledFn encode, CUtensorMap* m, const In& x, int64_t heads, int64_t width, int64_t L, int64_t Bsz, int dtype) {
    const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)Bsz};
    // the stride of a dimension of one is never used, but has to be valid
    const int64_t token = L > 1 ? x.token : heads * width, batch = Bsz > 1 ? x.batch : heads * width;
    const cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)token * 2, (cuuint64_t)batch * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)kChunk, 1}, step[4] = {1, 1, 1, 1};
    return encode(m, dtype == SS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x.p),
                  dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether these sizes may run on the tensor cores (their inputs too, if tc_input says so).
bool tc_sizes(int64_t L, int64_t N, int64_t P, int dtype) { return dtype != SS_F32 && N % 8 == 0 && P % 8 == 0 && L < (1ll << 31); }

// TMA's rules on an input: 16-byte units everywhere.
bool tc_input(const In& x, int64_t L, int64_t Bsz) {
    if (misaligned16(x.p)) return false;
    if (L > 1 && (x.token % 8 != 0 || x.token < 8 || x.token >= (1ll << 38))) return false;
    return Bsz <= 1 || (x.batch % 8 == 0 && x.batch >= 8 && x.batch < (1ll << 38));
}

// Segments that the walks over time are cut into: where there are fewer (batch row, head, value
// tile) units than SMs, or a last round of them leaves SMs idle.  Costs in chunks walked by one
// block: the walks themselves, the segments' sums before them (backward: of both directions), two a segment for the carry,
// four for the launches.  65536 tokens, 8 heads, N = P = 128: 792 us in 18 segments, 3664 whole; backward of 19362 tokens, 1 head,
// P 256: 326 and 1240.  (A cut has to be 5 % cheaper than the last one taken, so the cheapest of near ones is not always found.)
TcPlan tc_plan(int64_t heads, int64_t ptiles, int64_t chunks, bool backward) {
    const int64_t wide = backward ? 2 * ptiles : ptiles;  // both directions' walks
    auto rounds = [](int64_t blocks) { return ceil_div(blocks, kSms); };
    TcPlan best = {1, chunks};
    double least = (double)(rounds(heads * wide) * chunks);
    for (int64_t K = 2; K <= 128 && 2 * K <= chunks; K++) {
        const int64_t per = ceil_div(chunks, K);
        if (ceil_div(chunks, per) != K) continue;
        const int64_t sums = heads * (wide * (K - 1) + (backward ? K : K - 1));
        const double cost = (double)((rounds(heads * wide * K) + rounds(sums)) * per + 2 * K + 4);
        if (cost < 0.95 * least) {
            least = cost;
            best = {K, per};
        }
    }
    return best;
}

struct FwdTc {
    TcPlan plan;
    int64_t chunks;
    size_t keys, images, state, phi;
};
FwdTc fwdtc_layout(Layout& l, int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P) {
    FwdTc f;
    f.chunks = ceil_div(L, kChunk);
    f.plan = tc_plan(Bsz * H, ceil_div(P, kTileP), f.chunks, false);
    f.keys = l.take((size_t)Bsz * f.chunks * G * key_bytes(N));
    f.images = l.take((size_t)Bsz * H * f.chunks * kImageBytes);
    const bool cut = f.plan.K > 1;
    f.state = l.take(cut ? (size_t)Bsz * H * f.plan.K * N * P * 4 : 0);
    f.phi = l.take(cut ? (size_t)Bsz * H * f.plan.K * N * N * 4 : 0);
    return f;
}

// Blocks a group's heads are divided into by the first kernel: until there is one for each of four places on an SM.  37 tokens,
// 32 heads in 16 groups: 8.2 us, 12.0 undivided; 300 tokens, 64 heads in one: 11.5 and 231.  (Where there are nearly enough
// the parts' common products cost more than they bring: 2 x 1024 tokens, 32 heads in 8, N 64: 24.7 and 21.8.)
int prep_splits(int64_t blocks, int64_t rep) {
    int64_t s = ceil_div(4 * kSms, blocks);
    if (s > rep) s = rep;
    return (int)(s < 1 ? 1 : s);
}

// Forward on the tensor cores; *ran tells whether the inputs allow it.
int tc_forward(const Args& a, void* y, float* last, char* ws, cudaStream_t st, bool* ran) {
    *ran = false;
    if (!tc_sizes(a.L, a.N, a.P, a.dtype) || !tc_input(a.q, a.L, a.Bsz) || !tc_input(a.k, a.L, a.Bsz) || !tc_input(a.v, a.L, a.Bsz))
        return SS_OK;
    const auto encode = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!encode) return SS_OK;
    Layout l;
    const FwdTc f = fwdtc_layout(l, a.Bsz, a.L, a.H, a.G, a.N, a.P);
    TcWalkArgs w = {};
    PrepArgs p = {};
    const In yo = {y, a.H * a.P, a.L * a.H * a.P};
    if (!tc_map(encode, &p.q, a.q, a.G, a.N, a.L, a.Bsz, a.dtype) || !tc_map(encode, &p.k, a.k, a.G, a.N, a.L, a.Bsz, a.dtype) ||
        !tc_map(encode, &w.v, a.v, a.H, a.P, a.L, a.Bsz, a.dtype) || !tc_map(encode, &w.y, yo, a.H, a.P, a.L, a.Bsz, a.dtype))
        return SS_OK;
    const int rc = device_status_word(&w.status);
    if (rc != SS_OK) return rc;
    *ran = true;
    p.a = a;
    p.chunks = f.chunks;
    p.splits = prep_splits(a.Bsz * f.chunks * a.G, a.H / a.G);
    p.keys = ws + f.keys;
    p.images = ws + f.images;
    p.status = w.status;
    w.a = a;
    w.plan = f.plan;
    w.chunks = f.chunks;
    w.keys = p.keys;
    w.images = p.images;
    w.init = a.h0;
    w.last = last;
    w.seg_state = reinterpret_cast<float*>(ws + f.state);
    w.seg_phi = reinterpret_cast<float*>(ws + f.phi);
    w.yp = y;
    if (launch_prep(p, st) != cudaSuccess) return SS_ERR_CUDA;
    if (w.plan.K > 1 && (launch_tc_walk(w, kTcSum, st) != cudaSuccess || launch_tc_carry(w, nullptr, st) != cudaSuccess)) return SS_ERR_CUDA;
    return launch_tc_walk(w, kTcY, st) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

struct BwdTc {
    TcPlan plan;
    int64_t chunks;
    int splits;
    size_t starts, ends, phi, phi_t, keys, images, turned, before, after, us, xs, dys, before_inv, after_inv, u_inv, x_inv, dy_inv, dq, dk;
};
BwdTc bwdtc_layout(Layout& l, int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P) {
    BwdTc f;
    f.chunks = ceil_div(L, kChunk);
    f.splits = prep_splits(Bsz * f.chunks * G, H / G);
    f.plan = tc_plan(Bsz * H, ceil_div(P, kTileP), f.chunks, true);
    const size_t segs = f.plan.K > 1 ? (size_t)Bsz * H * f.plan.K : 0;
    for (size_t* x : {&f.starts, &f.ends}) *x = l.take(segs * N * P * 4);
    for (size_t* x : {&f.phi, &f.phi_t}) *x = l.take(segs * N * N * 4);
    const size_t heads = (size_t)Bsz * H * f.chunks, tiles = heads * ceil_div(P, kTileP);
    f.keys = l.take((size_t)Bsz * f.chunks * G * key_bytes(N));
    f.images = l.take(heads * kImageBytes);
    f.turned = l.take(heads * kTurnedBytes);
    f.before = l.take(tiles * state_bytes(N > 64 ? 2 : 1));
    f.after = l.take(tiles * state_bytes(N > 64 ? 2 : 1));
    f.us = l.take(tiles * kRowsBytes);
    f.xs = l.take(tiles * kRowsBytes);
    f.dys = l.take(tiles * kPieceBytes);
    for (size_t* x : {&f.before_inv, &f.after_inv, &f.u_inv, &f.x_inv, &f.dy_inv}) *x = l.take(tiles * 4);
    const size_t part = f.splits > 1 ? (size_t)f.splits * Bsz * L * G * N * 4 : 0;
    f.dq = l.take(part);
    f.dk = l.take(part);
    return f;
}

// Backward on the tensor cores; *ran tells whether the inputs allow it.
int tc_backward(const Args& a, const ss_gdr_bwd_desc& d, cudaStream_t st, bool* ran) {
    *ran = false;
    if (!tc_sizes(a.L, a.N, a.P, a.dtype) || !tc_input(a.q, a.L, a.Bsz) || !tc_input(a.k, a.L, a.Bsz) || !tc_input(a.v, a.L, a.Bsz) ||
        !tc_input(a.dy, a.L, a.Bsz))
        return SS_OK;
    const auto encode = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!encode) return SS_OK;
    Layout l;
    const BwdTc f = bwdtc_layout(l, a.Bsz, a.L, a.H, a.G, a.N, a.P);
    char* ws = static_cast<char*>(d.workspace);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    PrepArgs p = {};
    TcWalkArgs w = {};
    TcBackArgs r = {};
    TcChunkArgs c = {};
    if (!tc_map(encode, &p.q, a.q, a.G, a.N, a.L, a.Bsz, a.dtype) || !tc_map(encode, &p.k, a.k, a.G, a.N, a.L, a.Bsz, a.dtype) ||
        !tc_map(encode, &w.v, a.v, a.H, a.P, a.L, a.Bsz, a.dtype))
        return SS_OK;
    const int rc = device_status_word(&w.status);
    if (rc != SS_OK) return rc;
    *ran = true;
    p.a = a;
    p.chunks = f.chunks;
    p.splits = f.splits;
    p.keys = ws + f.keys;
    p.images = ws + f.images;
    p.turned = ws + f.turned;
    p.status = w.status;
    w.a = a;
    w.plan = f.plan;
    w.seg_state = f32(f.starts);
    w.seg_phi = f32(f.phi);
    w.seg_phi_t = f32(f.phi_t);
    r.seg_state = f32(f.ends);
    w.chunks = f.chunks;
    w.keys = p.keys;
    w.images = p.images;
    w.init = a.h0;
    w.states = ws + f.before;
    w.us = ws + f.us;
    w.state_inv = f32(f.before_inv);
    w.u_inv = f32(f.u_inv);
    r.init = a.dlast;
    r.last = d.dh0;
    r.states = ws + f.after;
    r.xs = ws + f.xs;
    r.state_inv = f32(f.after_inv);
    r.x_inv = f32(f.x_inv);
    r.turned = p.turned;
    r.dys = ws + f.dys;
    r.dy_inv = f32(f.dy_inv);
    c.a = a;
    c.chunks = f.chunks;
    c.splits = f.splits;
    c.keys = p.keys;
    c.images = p.images;
    c.before = w.states;
    c.after = r.states;
    c.us = w.us;
    c.xs = r.xs;
    c.dys = r.dys;
    c.before_inv = w.state_inv;
    c.after_inv = r.state_inv;
    c.u_inv = w.u_inv;
    c.x_inv = r.x_inv;
    c.dy_inv = r.dy_inv;
    c.dq = d.dq;
    c.dk = d.dk;
    c.dv = d.dv;
    c.dq_part = f32(f.dq);
    c.dk_part = f32(f.dk);
    c.dg = d.dg;
    c.dbeta = d.dbeta;
    c.status = w.status;
    if (launch_prep(p, st) != cudaSuccess || launch_dy(a, f.chunks, p.images, ws + f.dys, f32(f.dy_inv), st) != cudaSuccess) return SS_ERR_CUDA;
    if (w.plan.K > 1 && (launch_tc_sums(w, r, st) != cudaSuccess || launch_tc_carry(w, &r, st) != cudaSuccess)) return SS_ERR_CUDA;
    if (launch_tc_walks(w, r, st) != cudaSuccess || launch_tc_chunks(c, st) != cudaSuccess) return SS_ERR_CUDA;
    if (f.splits > 1 &&
        la::launch_sum_parts(c.dq_part, d.dq, c.dk_part, d.dk, f.splits, a.Bsz * a.L * a.G * a.N, a.dtype, st) != cudaSuccess)
        return SS_ERR_CUDA;
    return SS_OK;
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
    // the larger of what the two paths need: strides and pointers, which decide between them, are not known here
    Layout l, t;
    fwd32_layout(l, Bsz, L, H, N, P);
    if (tc_sizes(L, N, P, dtype)) fwdtc_layout(t, Bsz, L, H, G, N, P);
    return l.total > t.total ? l.total : t.total;
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
    bool ran;
    const int tc = tc_forward(a, d->y, d->last_state, static_cast<char*>(d->workspace), st, &ran);
    if (ran || tc != SS_OK) return tc;
    char* ws = static_cast<char*>(d->workspace);
    Layout l;
    const Fwd32 f = fwd32_layout(l, a.Bsz, a.L, a.H, a.N, a.P);
    WalkArgs w = {};
    w.a = a;
    Pairs* pairs = reinterpret_cast<Pairs*>(ws + f.pairs);
    w.pairs = pairs;
    w.init = a.h0;
    w.last = d->last_state;
    w.y = d->y;
    w.plan = f.plan;
    w.seg_state = reinterpret_cast<float*>(ws + f.starts);
    w.seg_phi = reinterpret_cast<float*>(ws + f.phi);
    if (launch_pairs(a, pairs, st) != cudaSuccess) return SS_ERR_CUDA;
    if (w.plan.K > 1 && launch_segments(w, nullptr, st) != cudaSuccess) return SS_ERR_CUDA;
    return launch_walk(w, st) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

size_t ss_gdr_bwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype) {
    if (check_sizes(Bsz, L, H, G, N, P, dtype) != SS_OK || empty(Bsz, L)) return 0;
    Layout l, t;
    bwd32_layout(l, Bsz, L, H, G, N, P);
    if (tc_sizes(L, N, P, dtype)) bwdtc_layout(t, Bsz, L, H, G, N, P);
    return l.total > t.total ? l.total : t.total;
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
    bool ran;
    const int tc = tc_backward(a, *d, st, &ran);
    if (ran || tc != SS_OK) return tc;
    char* ws = static_cast<char*>(d->workspace);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    Layout l;
    const Bwd32 bl = bwd32_layout(l, a.Bsz, a.L, a.H, a.G, a.N, a.P);
    WalkArgs keep = {}, back = {};
    keep.a = back.a = a;
    keep.chunks = back.chunks = bl.chunks;
    Pairs* pairs = reinterpret_cast<Pairs*>(ws + bl.pairs);
    keep.pairs = back.pairs = pairs;
    keep.init = a.h0;
    keep.rows = f32(bl.miss);
    keep.states = f32(bl.before);
    back.init = a.dlast;
    back.last = d->dh0;
    back.y = d->dv;
    back.rows = f32(bl.x);
    back.states = f32(bl.after);
    keep.plan = back.plan = bl.plan;
    keep.seg_state = f32(bl.starts);
    back.seg_state = f32(bl.ends);
    keep.seg_phi = back.seg_phi = f32(bl.phi);
    if (launch_pairs(a, pairs, st) != cudaSuccess) return SS_ERR_CUDA;
    if (bl.plan.K > 1 && launch_segments(keep, &back, st) != cudaSuccess) return SS_ERR_CUDA;
    if (launch_walks(keep, back, st) != cudaSuccess) return SS_ERR_CUDA;
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
    return (size_t)(norm_blocks(Bsz * L, Hq, Hk, N, kNormBlocks) + norm_blocks(Bsz * L, Hk, Hq, N, kNormBlocks)) * N * 4;
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
