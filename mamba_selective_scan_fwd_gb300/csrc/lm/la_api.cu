// C ABI of the linear attention and the gated group norm (include/ss_la.h).
// Everything is checked before the first CUDA call; on error nothing is
// written.
#include <cuda.h>

#include "la.h"
#include "la_tc.h"
#include "ss_la.h"

using namespace ss;
using namespace ss::la;

namespace {

bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int check_dtype(int dtype) { return dtype == SS_F32 || dtype == SS_F16 || dtype == SS_BF16 ? SS_OK : SS_ERR_UNSUPPORTED; }

int64_t elem(int dtype) { return dtype == SS_F32 ? 4 : 2; }

int check_sizes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype) {
    if (Bsz < 0 || L < 0 || H < 1 || G < 1 || N < 1 || P < 1 || H % G != 0) return SS_ERR_INVALID_PROBLEM;
    if (check_dtype(dtype) != SS_OK || N > kMaxN) return SS_ERR_UNSUPPORTED;
    // products stay inside int64, grids inside 2^31 - 1 blocks
    if (Bsz > (1 << 20) || L > (1ll << 31) || H > (1 << 16) || P > (1 << 16)) return SS_ERR_UNSUPPORTED;
    if (Bsz * H * ceil_div(P, 16) > (1ll << 24) || Bsz * L > (1ll << 36)) return SS_ERR_UNSUPPORTED;
    if (2 * Bsz * ceil_div(L, kChunk32) * H * ceil_div(P, kWalkP) >= (1ll << 31)) return SS_ERR_UNSUPPORTED;
    return SS_OK;
}

// A run of the workspace, in bytes from its start.
struct Layout {
    size_t total = 0;
    size_t take(size_t bytes) {
        const size_t at = total;
        total = align_up(total + bytes, 256);
        return at;
    }
};

// The FP32 path's workspace.
struct Walk32 {
    WalkPlan plan;
    size_t state, decay;
};
Walk32 walk32_layout(Layout& l, int64_t Bsz, int64_t L, int64_t H, int64_t N, int64_t P, int dirs) {
    Walk32 w;
    if (dirs == 1) w.plan = walk_plan(Bsz * H * ceil_div(P, kWalkP), L, N);
    else w.plan = {ceil_div(L, kChunk32), kChunk32};
    w.state = w.decay = 0;
    if (dirs == 2 || w.plan.K > 1) {
        w.state = l.take((size_t)dirs * Bsz * H * w.plan.K * N * P * 4);
        w.decay = l.take((size_t)dirs * Bsz * H * w.plan.K * 4);
    }
    return w;
}

struct Bwd32 {
    Walk32 walk;
    int64_t chunks;
    int splits;
    size_t dq, dk, dg, rows;
};
// Parts the heads of a group are divided into, so that the chunk kernel has
// about two blocks per SM (777 tokens, 16 heads in 4 groups: 44 us in four parts, 77 in
// one); each part beyond the first costs one more f32 copy of dq and dk.
int head_splits(int64_t blocks, int64_t rep) {
    int64_t s = ceil_div(2 * kSms, blocks);
    if (s > rep) s = rep;
    return (int)(s < 1 ? 1 : s);
}
Bwd32 bwd32_layout(Layout& l, int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P) {
    Bwd32 b;
    b.walk = walk32_layout(l, Bsz, L, H, N, P, 2);
    b.chunks = ceil_div(L, kChunk32);
    b.splits = head_splits(Bsz * b.chunks * G, H / G);
    const size_t part = b.splits > 1 ? (size_t)b.splits * Bsz * L * G * N * 4 : 0;
    b.dq = l.take(part);
    b.dk = l.take(part);
    b.dg = l.take((size_t)Bsz * L * H * 4);
    b.rows = l.take((size_t)kDgParts * H * 4);
    return b;
}

// ---------------------------------------------------------------- tensor-core path
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// [Bsz, L, heads, width] as a map {width, heads, L, Bsz}, boxes of 64 columns
// by 128 tokens in the 128-byte swizzle; what lies outside reads as zero.
// (f32: boxes of 32 columns)
bool tc_map(EncodeTiledFn encode, CUtensorMap* m, const In& x, int64_t heads, int64_t width, int64_t L, int64_t Bsz, int dtype) {
    const cuuint64_t esz = dtype == SS_F32 ? 4 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)Bsz};
    // the stride of a dimension of one is never used, but has to be valid
    const int64_t token = L > 1 ? x.token : heads * width, batch = Bsz > 1 ? x.batch : heads * width;
    const cuuint64_t strides[3] = {width * esz, token * esz, batch * esz};
    const cuuint32_t box[4] = {(cuuint32_t)(128 / esz), 1, (cuuint32_t)kChunkTc, 1}, step[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = dtype == SS_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == SS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode(m, type, 4,
                  const_cast<void*>(x.p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether these sizes may run on the tensor cores (their inputs too, if tc_input says
// so).  At every length: 37 tokens x 16 heads take 8.7 us so and 17.8 on the FP32 units,
// 4096 x 24 heads 47 and 250.
bool tc_sizes(int64_t L, int64_t N, int64_t P, int dtype) { return dtype != SS_F32 && N % 8 == 0 && P % 8 == 0 && L < (1ll << 31); }

// TMA's rules on an input: 16-byte units everywhere.
bool tc_input(const In& x, int64_t L, int64_t Bsz) {
    if (misaligned16(x.p)) return false;
    if (L > 1 && (x.token % 8 != 0 || x.token < 8 || x.token >= (1ll << 38))) return false;
    return Bsz <= 1 || (x.batch % 8 == 0 && x.batch >= 8 && x.batch < (1ll << 38));
}

struct WalkTc {
    TcPlan plan;
    size_t state, decay;
};
WalkTc walktc_layout(Layout& l, int64_t Bsz, int64_t L, int64_t H, int64_t N, int64_t P, int dirs, int64_t slots) {
    WalkTc w;
    w.plan = tc_plan(dirs * Bsz * H * ceil_div(P, kTileP), L, slots);
    w.state = l.take((size_t)w.plan.cut * w.plan.K * N * kTileP * 4);
    w.decay = l.take((size_t)w.plan.cut * w.plan.K * 4);
    return w;
}

// The sum pass of a walk cut in time, and the states its segments start from.
cudaError_t tc_carry(const TcWalkArgs& w, cudaStream_t st) {
    if (w.plan.cut == 0) return cudaSuccess;
    const cudaError_t e = launch_tc_state(w, true, st);
    return e != cudaSuccess ? e : launch_tc_carry(w, st);
}

// The forward's plans and the workspace of the larger: strides and pointers
// decide which path runs.
struct FwdPlan {
    Walk32 f32;
    WalkTc tc;
    size_t bytes;
};
FwdPlan fwd_plan(int64_t Bsz, int64_t L, int64_t H, int64_t N, int64_t P, int dtype) {
    FwdPlan p = {};
    Layout l, t;
    p.f32 = walk32_layout(l, Bsz, L, H, N, P, 1);
    if (tc_sizes(L, N, P, dtype)) p.tc = walktc_layout(t, Bsz, L, H, N, P, 1, 2 * kSms);
    p.bytes = l.total > t.total ? l.total : t.total;
    return p;
}

// Forward on the tensor cores; *ran tells whether the inputs allow it.
int tc_forward(const Args& a, const WalkTc& wl, void* y, float* last, char* ws, cudaStream_t st, bool* ran) {
    *ran = false;
    if (!tc_sizes(a.L, a.N, a.P, a.dtype) || !tc_input(a.q, a.L, a.Bsz) || !tc_input(a.k, a.L, a.Bsz) ||
        !tc_input(a.v, a.L, a.Bsz))
        return SS_OK;
    const auto encode = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!encode) return SS_OK;
    TcWalkArgs w = {};
    const In yo = {y, a.H * a.P, a.L * a.H * a.P};
    if (!tc_map(encode, &w.maps.q, a.q, a.G, a.N, a.L, a.Bsz, a.dtype) ||
        !tc_map(encode, &w.maps.k, a.k, a.G, a.N, a.L, a.Bsz, a.dtype) ||
        !tc_map(encode, &w.maps.v, a.v, a.H, a.P, a.L, a.Bsz, a.dtype) ||
        !tc_map(encode, &w.maps.y, yo, a.H, a.P, a.L, a.Bsz, a.dtype))
        return SS_OK;
    const int rc = device_status_word(&w.status);
    if (rc != SS_OK) return rc;
    w.a = a;
    w.plan = wl.plan;
    w.dirs = 1;
    w.dir[0] = {a.h0, last, nullptr, nullptr};
    w.seg_state = reinterpret_cast<float*>(ws + wl.state);
    w.seg_decay = reinterpret_cast<float*>(ws + wl.decay);
    *ran = true;
    if (tc_carry(w, st) != cudaSuccess) return SS_ERR_CUDA;
    return launch_tc_fwd(w, st) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

struct BwdTc {
    WalkTc walk;
    int64_t chunks, part_rows;
    int splits, dg_parts;
    size_t before, after, before_scale, after_scale, dq, dk, dg, rows;
};
BwdTc bwdtc_layout(Layout& l, int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype) {
    BwdTc b;
    b.walk = walktc_layout(l, Bsz, L, H, N, P, 2, kSms);
    b.chunks = ceil_div(L, kChunkTc);
    const int64_t ptiles = ceil_div(P, kTileP), states = Bsz * H * ptiles * b.chunks;
    const bool f16 = dtype == SS_F16;
    b.splits = f16 ? (int)(H / G * ptiles) : 1;
    b.dg_parts = f16 ? (int)ptiles : 1;
    const size_t images = (size_t)states * image_bytes(f16, N);
    b.before = l.take(images);
    b.after = l.take(images);
    b.before_scale = l.take(f16 ? states * 4 : 0);
    b.after_scale = l.take(f16 ? states * 4 : 0);
    b.part_rows = f16 ? (b.splits > 1 ? b.splits * Bsz : 0) : (H > G ? 2 * tc_bwd_blocks(Bsz * b.chunks * H) : 0);
    const size_t part = (size_t)b.part_rows * (f16 ? L * G : kChunkTc) * N * 4;
    b.dq = l.take(part);
    b.dk = l.take(part);
    b.dg = l.take((size_t)b.dg_parts * Bsz * L * H * 4);
    b.rows = l.take((size_t)kDgParts * H * 4);
    return b;
}

// What follows the chunk kernels of both paths: the parts' sums.
int bwd_sums(const ss_la_bwd_desc& d, int splits, const float* dq_part, const float* dk_part, const float* dg, int dg_parts, float* rows,
             cudaStream_t st) {
    if (splits > 1) {
        const int64_t n = d.Bsz * d.L * d.G * d.N;
        if (launch_sum_parts(dq_part, d.dq, dk_part, d.dk, splits, n, d.dtype, st) != cudaSuccess) return SS_ERR_CUDA;
    }
    if (d.g_per_head) {
        if (launch_sum_rows(dg, rows, d.dg, dg_parts * d.Bsz * d.L, d.H, st) != cudaSuccess) return SS_ERR_CUDA;
    } else if (dg_parts > 1) {
        if (launch_sum_parts(dg, d.dg, nullptr, nullptr, dg_parts, d.Bsz * d.L * d.H, SS_F32, st) != cudaSuccess) return SS_ERR_CUDA;
    }
    return SS_OK;
}

// Backward on the tensor cores; *ran tells whether the inputs allow it.
int tc_backward(const Args& a, const ss_la_bwd_desc& d, cudaStream_t st, bool* ran) {
    *ran = false;
    if (!tc_sizes(a.L, a.N, a.P, a.dtype) || !tc_input(a.q, a.L, a.Bsz) || !tc_input(a.k, a.L, a.Bsz) ||
        !tc_input(a.v, a.L, a.Bsz) || !tc_input(a.dy, a.L, a.Bsz))
        return SS_OK;
    const auto encode = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!encode) return SS_OK;
    TcWalkArgs w = {};
    TcBwdArgs b = {};
    char* ws = static_cast<char*>(d.workspace);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    Layout l;
    const BwdTc bl = bwdtc_layout(l, a.Bsz, a.L, a.H, a.G, a.N, a.P, a.dtype);
    const bool f16 = a.dtype == SS_F16;
    const int64_t part_heads = f16 ? a.G : 1, part_len = f16 ? a.L : kChunkTc;
    auto part = [&](size_t at) { return In{ws + at, part_heads * a.N, part_len * part_heads * a.N}; };
    const In dq = {d.dq, a.G * a.N, a.L * a.G * a.N}, dk = {d.dk, a.G * a.N, a.L * a.G * a.N},
             dv = {d.dv, a.H * a.P, a.L * a.H * a.P};
    if (!tc_map(encode, &b.maps.q, a.q, a.G, a.N, a.L, a.Bsz, a.dtype) ||
        !tc_map(encode, &b.maps.k, a.k, a.G, a.N, a.L, a.Bsz, a.dtype) ||
        !tc_map(encode, &b.maps.v, a.v, a.H, a.P, a.L, a.Bsz, a.dtype) ||
        !tc_map(encode, &b.maps.dy, a.dy, a.H, a.P, a.L, a.Bsz, a.dtype) ||
        !tc_map(encode, &b.maps.dq, dq, a.G, a.N, a.L, a.Bsz, a.dtype) ||
        !tc_map(encode, &b.maps.dk, dk, a.G, a.N, a.L, a.Bsz, a.dtype) ||
        (bl.part_rows > 0 &&
         (!tc_map(encode, &b.maps.dq_part, part(bl.dq), part_heads, a.N, part_len, bl.part_rows, SS_F32) ||
          !tc_map(encode, &b.maps.dk_part, part(bl.dk), part_heads, a.N, part_len, bl.part_rows, SS_F32))) ||
        !tc_map(encode, &b.maps.dv, dv, a.H, a.P, a.L, a.Bsz, a.dtype))
        return SS_OK;
    const int rc = device_status_word(&w.status);
    if (rc != SS_OK) return rc;
    *ran = true;
    w.maps.q = b.maps.q;
    w.maps.k = b.maps.k;
    w.maps.v = b.maps.v;
    w.maps.dy = b.maps.dy;
    w.a = a;
    w.plan = bl.walk.plan;
    w.seg_state = f32(bl.walk.state);
    w.seg_decay = f32(bl.walk.decay);
    w.chunks = bl.chunks;
    w.dirs = 2;
    w.dir[0] = {a.h0, nullptr, ws + bl.before, f32(bl.before_scale)};
    w.dir[1] = {a.dlast, d.dh0, ws + bl.after, f32(bl.after_scale)};
    if (tc_carry(w, st) != cudaSuccess || launch_tc_state(w, false, st) != cudaSuccess) return SS_ERR_CUDA;
    b.a = a;
    b.before = ws + bl.before;
    b.after = ws + bl.after;
    b.before_scale = f32(bl.before_scale);
    b.after_scale = f32(bl.after_scale);
    b.chunks = bl.chunks;
    const bool own_dg = !a.g_per_head && bl.dg_parts == 1;
    b.dg = own_dg ? d.dg : f32(bl.dg);
    b.splits = bl.splits;
    b.dq = d.dq;
    b.dk = d.dk;
    b.dq_part = f32(bl.dq);
    b.dk_part = f32(bl.dk);
    b.status = w.status;
    if (launch_tc_bwd(b, st) != cudaSuccess) return SS_ERR_CUDA;
    return bwd_sums(d, b.splits, b.dq_part, b.dk_part, b.dg, bl.dg_parts, f32(bl.rows), st);
}

bool empty(int64_t Bsz, int64_t L) { return Bsz == 0 || L == 0; }

// The state that no token changes: a copy of the incoming one, or zeros.
int pass_state(float* to, const float* from, int64_t Bsz, int64_t H, int64_t N, int64_t P, cudaStream_t st) {
    const size_t bytes = (size_t)Bsz * H * N * P * 4;
    if (!to || bytes == 0) return SS_OK;
    const cudaError_t e = from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st)
                               : cudaMemsetAsync(to, 0, bytes, st);
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

// The segments' sums and their carries.
cudaError_t start_states32(const WalkArgs& w, cudaStream_t st) {
    const cudaError_t e = launch_walk32(w, true, st);
    return e != cudaSuccess ? e : launch_carry32(w, st);
}

bool strides_ok(int64_t token, int64_t batch) { return token >= 0 && batch >= 0 && token <= (1ll << 40) && batch <= (1ll << 48); }

}  // namespace

extern "C" {

size_t ss_la_fwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype) {
    if (check_sizes(Bsz, L, H, G, N, P, dtype) != SS_OK || empty(Bsz, L)) return 0;
    return fwd_plan(Bsz, L, H, N, P, dtype).bytes;
}

int ss_la_fwd(const ss_la_fwd_desc* d, void* stream) {
    if (!d) return SS_ERR_INVALID_PROBLEM;
    const int rc = check_sizes(d->Bsz, d->L, d->H, d->G, d->N, d->P, d->dtype);
    if (rc != SS_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!strides_ok(d->q_token, d->q_batch) || !strides_ok(d->k_token, d->k_batch) || !strides_ok(d->v_token, d->v_batch))
        return SS_ERR_INVALID_PROBLEM;
    if (misaligned16(d->y) || misaligned16(d->h0) || misaligned16(d->last_state) || misaligned16(d->workspace))
        return SS_ERR_UNSUPPORTED;
    if (empty(d->Bsz, d->L)) return pass_state(d->last_state, d->h0, d->Bsz, d->H, d->N, d->P, st);
    if (!d->q || !d->k || !d->v || !d->g || !d->y) return SS_ERR_INVALID_PROBLEM;
    const FwdPlan plan = fwd_plan(d->Bsz, d->L, d->H, d->N, d->P, d->dtype);
    const size_t need = plan.bytes;
    if (d->workspace_bytes < need || (need > 0 && !d->workspace)) return SS_ERR_WORKSPACE_TOO_SMALL;
    Args a = {};
    a.q = {d->q, d->q_token, d->q_batch};
    a.k = {d->k, d->k_token, d->k_batch};
    a.v = {d->v, d->v_token, d->v_batch};
    a.g = d->g;
    a.h0 = d->h0;
    a.lengths = d->lengths;
    a.Bsz = d->Bsz; a.L = d->L; a.H = d->H; a.G = d->G; a.N = d->N; a.P = d->P;
    a.scale = d->scale;
    a.dtype = d->dtype;
    a.g_per_head = d->g_per_head ? 1 : 0;
    char* ws = static_cast<char*>(d->workspace);
    bool ran;
    const int tc = tc_forward(a, plan.tc, d->y, d->last_state, ws, st, &ran);
    if (ran || tc != SS_OK) return tc;
    const Walk32& wl = plan.f32;
    WalkArgs w = {};
    w.a = a;
    w.plan = wl.plan;
    w.dirs = 1;
    w.dir[0] = {a.h0, d->last_state};
    w.seg_state = reinterpret_cast<float*>(ws + wl.state);
    w.seg_decay = reinterpret_cast<float*>(ws + wl.decay);
    w.y = d->y;
    if (w.plan.K > 1 && start_states32(w, st) != cudaSuccess) return SS_ERR_CUDA;
    return launch_walk32(w, false, st) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

size_t ss_la_bwd_workspace_bytes(int64_t Bsz, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P, int dtype) {
    if (check_sizes(Bsz, L, H, G, N, P, dtype) != SS_OK || empty(Bsz, L)) return 0;
    Layout l, t;
    bwd32_layout(l, Bsz, L, H, G, N, P);
    if (tc_sizes(L, N, P, dtype)) bwdtc_layout(t, Bsz, L, H, G, N, P, dtype);
    return l.total > t.total ? l.total : t.total;
}

int ss_la_bwd(const ss_la_bwd_desc* d, void* stream) {
    if (!d) return SS_ERR_INVALID_PROBLEM;
    const int rc = check_sizes(d->Bsz, d->L, d->H, d->G, d->N, d->P, d->dtype);
    if (rc != SS_OK) return rc;
    if ((d->h0 == nullptr) != (d->dh0 == nullptr)) return SS_ERR_INVALID_PROBLEM;
    if (!strides_ok(d->q_token, d->q_batch) || !strides_ok(d->k_token, d->k_batch) ||
        !strides_ok(d->v_token, d->v_batch) || !strides_ok(d->dy_token, d->dy_batch))
        return SS_ERR_INVALID_PROBLEM;
    const void* ptrs[] = {d->h0, d->dlast_state, d->dq, d->dk, d->dv, d->dg, d->dh0, d->workspace};
    for (const void* p : ptrs)
        if (misaligned16(p)) return SS_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (empty(d->Bsz, d->L)) {
        if (d->g_per_head) {
            if (!d->dg) return SS_ERR_INVALID_PROBLEM;
            if (cudaMemsetAsync(d->dg, 0, (size_t)d->H * 4, st) != cudaSuccess) return SS_ERR_CUDA;
        }
        return pass_state(d->dh0, d->dlast_state, d->Bsz, d->H, d->N, d->P, st);
    }
    if (!d->q || !d->k || !d->v || !d->g || !d->dy || !d->dq || !d->dk || !d->dv || !d->dg) return SS_ERR_INVALID_PROBLEM;
    const size_t need = ss_la_bwd_workspace_bytes(d->Bsz, d->L, d->H, d->G, d->N, d->P, d->dtype);
    if (d->workspace_bytes < need || !d->workspace) return SS_ERR_WORKSPACE_TOO_SMALL;
    Args a = {};
    a.q = {d->q, d->q_token, d->q_batch};
    a.k = {d->k, d->k_token, d->k_batch};
    a.v = {d->v, d->v_token, d->v_batch};
    a.dy = {d->dy, d->dy_token, d->dy_batch};
    a.g = d->g;
    a.h0 = d->h0;
    a.dlast = d->dlast_state;
    a.lengths = d->lengths;
    a.Bsz = d->Bsz; a.L = d->L; a.H = d->H; a.G = d->G; a.N = d->N; a.P = d->P;
    a.scale = d->scale;
    a.dtype = d->dtype;
    a.g_per_head = d->g_per_head ? 1 : 0;
    bool ran;
    const int tc = tc_backward(a, *d, st, &ran);
    if (ran || tc != SS_OK) return tc;
    char* ws = static_cast<char*>(d->workspace);
    Layout l;
    const Bwd32 bl = bwd32_layout(l, a.Bsz, a.L, a.H, a.G, a.N, a.P);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    WalkArgs w = {};
    w.a = a;
    w.plan = bl.walk.plan;
    w.seg_state = f32(bl.walk.state);
    w.seg_decay = f32(bl.walk.decay);
    w.dirs = 2;
    w.dir[0] = {a.h0, nullptr};
    w.dir[1] = {a.dlast, d->dh0};
    if (start_states32(w, st) != cudaSuccess) return SS_ERR_CUDA;
    BwdArgs b = {};
    b.a = a;
    b.before = w.seg_state;
    b.after = w.seg_state + a.Bsz * a.H * bl.chunks * a.N * a.P;
    b.chunks = bl.chunks;
    b.dq = d->dq; b.dk = d->dk; b.dv = d->dv;
    b.dg = a.g_per_head ? f32(bl.dg) : d->dg;
    b.dq_part = f32(bl.dq);
    b.dk_part = f32(bl.dk);
    b.splits = bl.splits;
    if (launch_bwd32(b, st) != cudaSuccess) return SS_ERR_CUDA;
    return bwd_sums(*d, b.splits, b.dq_part, b.dk_part, b.dg, 1, f32(bl.rows), st);
}

int ss_la_step(const ss_la_step_desc* d, void* stream) {
    if (!d) return SS_ERR_INVALID_PROBLEM;
    const int rc = check_sizes(d->Bsz, 1, d->H, d->G, d->N, d->P, d->dtype);
    if (rc != SS_OK) return rc;
    if (d->pool < 0 || (!d->slots && d->pool < d->Bsz) || d->q_batch < 0 || d->k_batch < 0 || d->v_batch < 0)
        return SS_ERR_INVALID_PROBLEM;
    if (misaligned16(d->state) || misaligned16(d->y)) return SS_ERR_UNSUPPORTED;
    if (d->Bsz == 0) return SS_OK;
    if (!d->q || !d->k || !d->v || !d->g || !d->y || (!d->state && d->pool > 0)) return SS_ERR_INVALID_PROBLEM;
    StepArgs s = {d->q, d->k, d->v, d->g, d->state, d->slots, d->y, d->q_batch, d->k_batch, d->v_batch,
                  d->Bsz, d->H, d->G, d->N, d->P, d->pool, d->scale, d->dtype, d->g_per_head ? 1 : 0};
    return launch_step(s, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

int ss_la_selftest_wait_timeout(int64_t limit_ns, void* stream) {
    if (limit_ns < 0 || limit_ns > (int64_t)kWaitLimitNs) return SS_ERR_INVALID_PROBLEM;
    int* status = nullptr;
    const int rc = device_status_word(&status);
    if (rc != SS_OK) return rc;
    return launch_late_timeout(status, (uint64_t)limit_ns, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

namespace {
int check_gnorm(int64_t M, int64_t C, int64_t groups, float eps, int flags, int dtype, bool z) {
    if (M < 0 || C < 1 || groups < 1 || C % groups != 0 || !(eps >= 0.0f)) return SS_ERR_INVALID_PROBLEM;
    if (flags & ~(SS_GNORM_CENTER | SS_GNORM_GATE_FIRST)) return SS_ERR_INVALID_PROBLEM;
    if ((flags & SS_GNORM_GATE_FIRST) && !z) return SS_ERR_INVALID_PROBLEM;
    if (check_dtype(dtype) != SS_OK || C / groups > 8192 || C > (1 << 24) || M > (1ll << 36)) return SS_ERR_UNSUPPORTED;
    return SS_OK;
}
}  // namespace

int ss_gnorm_fwd(const void* x, const float* weight, const float* bias, const void* z, void* out, int64_t M, int64_t C,
                 int64_t groups, float eps, int flags, int dtype, void* stream) {
    const int rc = check_gnorm(M, C, groups, eps, flags, dtype, z != nullptr || M == 0);
    if (rc != SS_OK) return rc;
    if (M == 0) return SS_OK;
    if (!x || !out) return SS_ERR_INVALID_PROBLEM;
    GnormArgs a = {};
    a.x = x; a.z = z; a.weight = weight; a.bias = bias; a.out = out;
    a.M = M; a.C = C; a.groups = groups;
    a.eps = eps; a.flags = flags; a.dtype = dtype;
    return launch_gnorm_fwd(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

size_t ss_gnorm_bwd_workspace_bytes(int64_t M, int64_t C, int64_t groups, int dtype) {
    if (check_gnorm(M, C, groups, 0.0f, 0, dtype, true) != SS_OK) return 0;
    return (size_t)gnorm_bwd_blocks(M, C, groups) * 2 * C * 4;
}

int ss_gnorm_bwd(const void* x, const float* weight, const float* bias, const void* z, const void* dout, void* dx,
                 void* dz, float* dweight, float* dbias, int64_t M, int64_t C, int64_t groups, float eps, int flags,
                 int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_gnorm(M, C, groups, eps, flags, dtype, z != nullptr || M == 0);
    if (rc != SS_OK) return rc;
    if ((weight == nullptr) != (dweight == nullptr) || (bias == nullptr) != (dbias == nullptr)) return SS_ERR_INVALID_PROBLEM;
    if (M > 0 && (!x || !dout || !dx || (z == nullptr) != (dz == nullptr))) return SS_ERR_INVALID_PROBLEM;
    if (misaligned16(workspace)) return SS_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < ss_gnorm_bwd_workspace_bytes(M, C, groups, dtype)) return SS_ERR_WORKSPACE_TOO_SMALL;
    GnormArgs a = {};
    a.x = x; a.z = z; a.dout = dout; a.weight = weight; a.bias = bias;
    a.dx = dx; a.dz = dz; a.dweight = dweight; a.dbias = dbias;
    a.part = static_cast<float*>(workspace);
    a.M = M; a.C = C; a.groups = groups;
    a.eps = eps; a.flags = flags; a.dtype = dtype;
    return launch_gnorm_bwd(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

}  // extern "C"
