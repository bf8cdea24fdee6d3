// Gated delta rule on the FP32 units: every io type, any N <= 128, P and strides.
// f32 inputs run here, and 16-bit inputs that the tensor-core path's rules exclude.
//
// Forward: the recurrence itself, four tokens at a time.  The columns of the state (value
// channels) are independent, so a column's N values lie in the registers of N / 16
// lanes.  Backward: with x_t = R_t^T k_t, R_t the adjoint of S_t,
//   R_t = (adjoint left by t + 1) + scale q_t dy_t^T,   adjoint left = e^{g_t} (R_t - beta_t k_t x_t^T)
// a second walk of the same form from the last token gives x and the adjoints R at
// the chunks' ends, the forward's walk the misses w_t = v_t - e^{g_t} S^T k_t
// (u = beta w) and the states H at their starts.  With u and x known everything else
// is products inside a chunk of 64 tokens (c_i: cumulative log decay, cl: its end):
//   E_ij = scale e^{c_i - c_j} dy_i . u_j (j <= i),   F_ij = -beta_i e^{c_i - c_j} x_i . u_j (j < i)
//   dq_i = scale e^{c_i} H dy_i + sum_j E_ij k_j
//   dk_i = -beta_i e^{c_i} H x_i + sum_j F_ij k_j + e^{cl - c_i} R u_i + sum_j (E_ji q_j + F_ji k_j)
//   dv_i = beta_i x_i,   dbeta_i = x_i . w_i
//   dg_t = every path that crosses token t, by its two ends: sum_{i >= t} a_i + sum_{j < t} b_j
//          + sum_{j < t <= i} (E_ij q_i . k_j + F_ij k_i . k_j) + e^{cl} <R, H>
// a_i, b_j: the parts of q_i . dq_i + k_i . dk_i that come from H, of k_j . dk_j that go to R.
#include "../simd.cuh"
#include "gdr_dev.cuh"

namespace ss {
namespace gdr {
namespace {

using la::Decay;
using la::Two;
using la::two_diff;

__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// 16 bytes on their way to shared memory, or zeros
__device__ __forceinline__ void copy16(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <int LN> __device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int o = LN / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// One block: 16 tokens of one head, thread (token t, j of its four, which product).
template <typename T> __global__ void __launch_bounds__(128) k_pairs(Args a, Pairs* pairs, int64_t tiles) {
    constexpr int TT = kWalkT, LD = la::kMaxN + 4;
    __shared__ __align__(16) float s_k[TT][LD], s_q[TT][LD];
    __shared__ float s_g[TT];
    const int tid = threadIdx.x, lane = tid & 31, N = (int)a.N, NP = (N + 3) & ~3;
    int64_t id = blockIdx.x;
    const int64_t tile = id % tiles;
    id /= tiles;
    const int64_t h = id % a.H, b = id / a.H, hq = h / (a.H / a.G), t0 = tile * TT;
    const int nv = (int)max((int64_t)0, min((int64_t)TT, row_length(a, b) - t0));
    if (nv == 0) return;
    const T* kp = static_cast<const T*>(a.k.p) + b * a.k.batch + t0 * a.k.token + hq * a.N;
    const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + t0 * a.q.token + hq * a.N;
    Pairs* to = pairs + blockIdx.x;
#pragma unroll 4
    for (int i = tid; i < TT * la::kMaxN; i += 128) {
        const int t = i / la::kMaxN, n = i % la::kMaxN;
        if (n >= NP) continue;
        const bool on = t < nv && n < N;
        s_k[t][n] = on ? ldf(kp + t * a.k.token + n) : 0.0f;
        s_q[t][n] = on ? a.scale * ldf(qp + t * a.q.token + n) : 0.0f;
    }
    if (tid < 32) {  // decays inside a four: sums of at most four numbers
        const float g = lane < nv ? log_decay(a, b, t0 + lane, h) : 0.0f;
        const int f = lane & 3;
        float up = g, down = 0.0f;
#pragma unroll
        for (int o = 1; o < 4; o++) {
            const float before = __shfl_up_sync(kFull, g, o), after = __shfl_down_sync(kFull, g, o);
            if (o <= f) up += before;
            if (o <= 3 - f) down += after;
        }
        if (lane < TT) {
            s_g[lane] = g;
            to->up[lane] = expf(up);
            to->down[lane] = expf(down);
            to->beta[lane] = lane < nv ? a.beta[(b * a.L + t0 + lane) * a.H + h] : 0.0f;
            if (f == 3) {
                const Decay d = la::decay_of(up);
                to->by[lane >> 2] = d.by;
                to->weak[lane >> 2] = d.weak;
            }
        }
    }
    __syncthreads();
    const int t = tid >> 3, j = tid >> 1 & 3, o = t & ~3, f = t & 3;
    const bool is_q = tid & 1;
    const float *x = is_q ? s_q[t] : s_k[t], *y = s_k[o + j];
    float s[4] = {};
#pragma unroll 4
    for (int n = 0; n < NP; n += 4) {
        const float4 u = at4(x + n), v = at4(y + n);
        s[0] = fmaf(u.x, v.x, s[0]);
        s[1] = fmaf(u.y, v.y, s[1]);
        s[2] = fmaf(u.z, v.z, s[2]);
        s[3] = fmaf(u.w, v.w, s[3]);
    }
    float c = 0.0f;
#pragma unroll
    for (int e = 1; e < 4; e++)
        if (e > j && e <= f) c += s_g[o + e];
    (is_q ? to->qk : to->kk)[t][j] = j <= f ? expf(c) * ((s[0] + s[1]) + (s[2] + s[3])) : 0.0f;
}

// One block: 64 / LN value channels of one head, one a lane and LN lanes a channel; lane ln of a
// channel holds the states n = 4 (ln + LN j) + e, j, e < 4, in pairs of e (runs of four so that the
// lanes' reads of k and q are 16 bytes side by side; those reads, four cycles of shared memory each, are
// what bounds an SM's blocks, so blocks are small and spread).  Tokens go by fours, whose products with the
// old state do not wait for one another:
//   miss_t = v_t - e^{c_t} S^T k_t - sum_{j < t} e^{c_t - c_j} (k_t . k_j) u_j,   u_t = beta_t miss_t
//   y_t = e^{c_t} S^T q_t + sum_{j <= t} e^{c_t - c_j} (q_t . k_j) u_j,   S <- e^{cl} S + sum_j e^{cl - c_j} k_j u_j^T
// so that a chain of sums over the lanes is paid once for four tokens.  The backward's walk is the same from
// the other end.  2 x 1000 tokens, 24 heads, N = P = 64: 143 us beside 17 for the pairs' products (token by token 228;
// with four interleaved chains of sums and q held in registers 149).
//
// Few heads of many tokens are cut into segments (walk_plan): the same walk takes their sums, whose columns (N of Phi, P of E)
// are as independent, a carry joins them, and the walk proper starts from what it left.  Backward of 777 tokens, 16 heads, N 32,
// P 64: 92 us in one piece, sums 30, carry 7 and walks 32 in four.
template <int LN, WalkMode MODE> struct WalkStage {
    static constexpr bool Q = MODE != kWalkSum && MODE != kWalkKeep;
    float k[kWalkT][16 * LN], q[Q ? kWalkT : 1][16 * LN], v[kWalkT][64 / LN];
    Pairs p;
};
// phi (kWalkSum): from the identity without v, else from zero
template <typename T, int LN, WalkMode MODE> __device__ __forceinline__ void walk(const WalkArgs& w, int64_t id, bool phi = false) {
    using Stage = WalkStage<LN, MODE>;
    constexpr bool SUM = MODE == kWalkSum, BACK = MODE == kWalkBack || MODE == kWalkBackSum, NOQ = !Stage::Q;
    constexpr int NT = 64, NP = 16 * LN, PT = NT / LN, TT = kWalkT;
    extern __shared__ __align__(16) char smem[];
    Stage* s_stage = reinterpret_cast<Stage*>(smem);
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, ln = lane % LN;
    const int64_t width = phi ? a.N : a.P, ptiles = (a.P + PT - 1) / PT, tiles_of = phi ? (a.N + PT - 1) / PT : ptiles;
    const int64_t p0 = (id % tiles_of) * PT;
    id /= tiles_of;
    const int64_t seg = id % w.plan.K;
    id /= w.plan.K;
    const int64_t h = id % a.H, b = id / a.H, hq = h / (a.H / a.G), bh = b * a.H + h;
    const int N = (int)a.N, pleft = (int)min((int64_t)PT, width - p0);
    const int col = tid / LN;  // of the block's channels
    const int64_t len = row_length(a, b), NPel = a.N * a.P;
    const In& vin = BACK ? a.dy : a.v;
    const T* kp = static_cast<const T*>(a.k.p) + b * a.k.batch + hq * a.N;
    const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + hq * a.N;
    const T* vp = static_cast<const T*>(vin.p) + b * vin.batch + h * a.P + (phi ? 0 : p0);
    const int64_t all_tiles = (a.L + TT - 1) / TT;

    float2 S[8];  // [2 j + e / 2]
    auto state = [&](float* p, bool put) {  // p: the head's N x P
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int n = 4 * (ln + LN * (i / 2)) + 2 * (i & 1);
            const bool ok = p && col < pleft;
            float* q = p + n * width + p0 + col;
            if (put) {
                if (ok && n < N) q[0] = S[i].x;
                if (ok && n + 1 < N) q[width] = S[i].y;
            } else {
                S[i].x = ok && n < N ? q[0] : 0.0f;
                S[i].y = ok && n + 1 < N ? q[width] : 0.0f;
            }
        }
    };
    float* const seg_state = w.plan.K > 1 ? w.seg_state + (bh * w.plan.K + seg) * NPel : nullptr;
    if (phi) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int64_t n = 4 * (ln + LN * (i / 2)) + 2 * (i & 1), c = p0 + col;
            S[i] = make_float2(n == c ? 1.0f : 0.0f, n + 1 == c ? 1.0f : 0.0f);
        }
    } else {
        state(SUM || MODE == kWalkBackSum ? nullptr : seg_state ? seg_state : w.init ? const_cast<float*>(w.init) + bh * NPel : nullptr, false);
    }

    const int64_t first = seg * w.plan.seg, tiles = max((int64_t)0, min((len + TT - 1) / TT, first + w.plan.seg) - first);
    auto start = [&](int64_t i) { return (first + (BACK ? tiles - 1 - i : i)) * TT; };
    auto fetch = [&](int64_t i) {
        Stage& s = s_stage[i & 1];
        const int64_t t0 = start(i);
        const int nv = (int)min((int64_t)TT, len - t0);
        const char* pairs = reinterpret_cast<const char*>(w.pairs + bh * all_tiles + t0 / TT);
        if (tid < (int)sizeof(Pairs) / 16) copy16(reinterpret_cast<char*>(&s.p) + 16 * tid, pairs + 16 * tid, true);
        if (w.vec) {
#pragma unroll
            for (int e = 0; e < TT * NP / 4 / NT; e++) {
                const int x = tid + NT * e, t = x / (NP / 4), n = x % (NP / 4) * 4;
                const bool on = t < nv && n < N;
                const int64_t tt = on ? t0 + t : 0;
                copy16(&s.k[t][n], kp + tt * a.k.token + (on ? n : 0), on);
                if (!NOQ) copy16(&s.q[t][n], qp + tt * a.q.token + (on ? n : 0), on);
            }
#pragma unroll
            for (int e = 0; e < (TT * PT / 4 + NT - 1) / NT; e++) {
                const int x = tid + NT * e, t = x / (PT / 4), c = x % (PT / 4) * 4;
                if (t >= TT) break;
                const bool on = !phi && t < nv && c < pleft;
                copy16(&s.v[t][c], vp + (on ? t0 + t : 0) * vin.token + (on ? c : 0), on);
            }
        } else {
#pragma unroll 4
            for (int x = tid; x < TT * NP; x += NT) {
                const int t = x / NP, n = x % NP;
                const bool on = t < nv && n < N;
                s.k[t][n] = on ? ldf(kp + (t0 + t) * a.k.token + n) : 0.0f;
                if (!NOQ) s.q[t][n] = on ? ldf(qp + (t0 + t) * a.q.token + n) : 0.0f;
            }
#pragma unroll 4
            for (int x = tid; x < TT * PT; x += NT) {
                const int t = x / PT, c = x % PT;
                s.v[t][c] = !phi && t < nv && c < pleft ? ldf(vp + (t0 + t) * vin.token + c) : 0.0f;
            }
        }
        copy_commit();
    };
    auto read = [&](const float* from, float2 (&x)[8]) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float4 v = at4(from + 4 * (ln + LN * j));
            x[2 * j] = make_float2(v.x, v.y);
            x[2 * j + 1] = make_float2(v.z, v.w);
        }
    };
    auto dot = [&](const float2 (&x)[8]) {
        float2 s[2] = {};
#pragma unroll
        for (int j = 0; j < 8; j++) s[j & 1] = fma2(x[j], S[j], s[j & 1]);
        s[0] = add2(s[0], s[1]);
        return s[0].x + s[0].y;
    };
    if (tiles > 0) fetch(0);
    for (int64_t i = 0; i < tiles; i++) {
        const int64_t t0 = start(i);
        const int nv = (int)min((int64_t)TT, len - t0);
        const Stage& s = s_stage[i & 1];
        copy_wait();
        __syncthreads();  // (and: the stage before is read)
        if (i + 1 < tiles) fetch(i + 1);
        // the state before a chunk's first token, the adjoint after its last one
        if (MODE == kWalkKeep ? t0 % kChunk == 0 : MODE == kWalkBack && (i == 0 || (t0 + TT) % kChunk == 0))
            state(w.states + (bh * w.chunks + t0 / kChunk) * NPel, true);
        const int fours = (nv + 3) >> 2;
        const int64_t row0 = ((b * a.L + t0) * a.H + h) * a.P + p0 + col;
#pragma unroll 1
        for (int u = 0; u < fours; u++) {
            const int o = kFour * (BACK ? fours - 1 - u : u);
            float2 k[kFour][8];
            float ks[kFour], qs[kFour];
#pragma unroll
            for (int t = 0; t < kFour; t++) {
                read(s.k[o + t], k[t]);
                ks[t] = dot(k[t]);
            }
            if (MODE == kWalkY)
#pragma unroll
                for (int t = 0; t < kFour; t++) {
                    float2 q[8];
                    read(s.q[o + t], q);
                    qs[t] = dot(q);
                }
#pragma unroll
            for (int r = LN / 2; r > 0; r >>= 1)
#pragma unroll
                for (int t = 0; t < kFour; t++) {
                    ks[t] += __shfl_xor_sync(kFull, ks[t], r);
                    if (MODE == kWalkY) qs[t] += __shfl_xor_sync(kFull, qs[t], r);
                }
            float v[kFour], x[kFour], kk[kFour][kFour], qk[kFour][kFour], up[kFour], down[kFour], beta[kFour];
            auto row = [](float (&to)[kFour], const float* from) {
                const float4 f = at4(from);
                to[0] = f.x;
                to[1] = f.y;
                to[2] = f.z;
                to[3] = f.w;
            };
#pragma unroll
            for (int t = 0; t < kFour; t++) {
                v[t] = s.v[o + t][col];
                if (t > 0) row(kk[t], s.p.kk[o + t]);
                if (!NOQ) row(qk[t], s.p.qk[o + t]);
            }
            row(up, &s.p.up[o]);
            row(down, &s.p.down[o]);
            row(beta, &s.p.beta[o]);
            const float by = s.p.by[o >> 2];
            const bool weak = s.p.weak[o >> 2];
            if (BACK) {
#pragma unroll
                for (int t = kFour - 1; t >= 0; t--) {
                    float z = down[t] * ks[t];
#pragma unroll
                    for (int e = t; e < kFour; e++) z = fmaf(qk[e][t], v[e], z);
#pragma unroll
                    for (int e = kFour - 1; e > t; e--) z = fmaf(-beta[e] * kk[e][t], x[e], z);
                    x[t] = z;
                }
            } else {
                float us[kFour];
#pragma unroll
                for (int t = 0; t < kFour; t++) {
                    float z = fmaf(-up[t], ks[t], v[t]);
#pragma unroll
                    for (int e = 0; e < t; e++) z = fmaf(-kk[t][e], us[e], z);
                    x[t] = z;
                    us[t] = beta[t] * z;
                }
#pragma unroll
                for (int t = 0; t < kFour; t++) ks[t] = down[t] * us[t];  // what enters the state
                if (MODE == kWalkY)
#pragma unroll
                    for (int t = 0; t < kFour; t++) {
                        float z = a.scale * up[t] * qs[t];
#pragma unroll
                        for (int e = 0; e <= t; e++) z = fmaf(qk[t][e], us[e], z);
                        x[t] = z;
                    }
            }
            if (weak) {
#pragma unroll
                for (int j = 0; j < 8; j++) S[j] = fma2(splat2(by), S[j], S[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++) S[j] = mul2(splat2(by), S[j]);
            }
#pragma unroll
            for (int t = 0; t < kFour; t++) {
                const float2 f = splat2(BACK ? -up[t] * beta[t] * x[t] : ks[t]);
#pragma unroll
                for (int j = 0; j < 8; j++) S[j] = fma2(k[t][j], f, S[j]);
                if (BACK) {
                    float2 q[8];
                    read(s.q[o + t], q);
                    const float2 y = splat2(a.scale * up[t] * v[t]);
#pragma unroll
                    for (int j = 0; j < 8; j++) S[j] = fma2(q[j], y, S[j]);
                }
            }
            if (MODE != kWalkSum && MODE != kWalkBackSum && ln == 0 && col < pleft)
#pragma unroll
                for (int t = 0; t < kFour; t++)
                    if (o + t < nv) {
                        const int64_t to = row0 + (o + t) * a.H * a.P;
                        if (MODE != kWalkY) w.rows[to] = x[t];
                        if (MODE != kWalkKeep) st(static_cast<T*>(w.y) + to, MODE == kWalkBack ? beta[t] * x[t] : x[t]);
                    }
        }
    }
    if (MODE == kWalkY || MODE == kWalkBack)  // rows that do not count
        for (int64_t t = max(len, first * TT) + tid / 32; t < min(a.L, (first + w.plan.seg) * TT); t += NT / 32)
            for (int c = lane; c < pleft; c += 32) st(static_cast<T*>(w.y) + ((b * a.L + t) * a.H + h) * a.P + p0 + c, 0.0f);
    if (phi) state(w.seg_phi + (bh * w.plan.K + seg) * a.N * a.N, true);
    else if (SUM || MODE == kWalkBackSum) state(seg_state, true);
    else if (w.last && seg == (BACK ? 0 : w.plan.K - 1)) state(w.last + bh * NPel, true);
}
// FIT blocks an SM: left alone the walk takes 200 registers and more and four blocks fit; held to six it is 2 to 3 % slower where
// there are few, and from five on faster (112 tokens, N = P = 128, four blocks an SM 30.6 and 31.3 us, six 59.5 and 39.7).
template <typename T, int LN, int FIT> __global__ void __launch_bounds__(64, FIT) k_walk(WalkArgs w) { walk<T, LN, kWalkY>(w, blockIdx.x); }
template <typename T, int LN, int FIT> __global__ void __launch_bounds__(64, FIT) k_walks(WalkArgs keep, WalkArgs back) {
    if (blockIdx.y == 0) walk<T, LN, kWalkKeep>(keep, blockIdx.x);
    else walk<T, LN, kWalkBack>(back, blockIdx.x);
}
// blockIdx.y: 0 Phi, 1 E, 2 E'.  Nothing follows the last segment, nothing comes before the first.
template <typename T, int LN> __global__ void __launch_bounds__(64, 6) k_sums(WalkArgs w, WalkArgs back) {
    constexpr int PT = 64 / LN;
    const int64_t wide = ((blockIdx.y == 0 ? w.a.N : w.a.P) + PT - 1) / PT, K = w.plan.K, seg = blockIdx.x / wide % K;
    if (blockIdx.x >= wide * K * w.a.H * w.a.Bsz) return;
    if (blockIdx.y == 2 ? seg == 0 : seg == K - 1 && (blockIdx.y == 1 || gridDim.y == 2)) return;
    if (blockIdx.y < 2) walk<T, LN, kWalkSum>(w, blockIdx.x, blockIdx.y == 0);
    else walk<T, LN, kWalkBackSum>(back, blockIdx.x);
}

// S <- Phi S + E over the segments from the first (blockIdx.y 0), R <- Phi^T R + E' from the last (1); the sums' places receive
// what each segment starts from.  A block: 8 columns of one head, two threads a state; the next Phi is on its way while
// one is used.
constexpr int kCarryCols = 8;
__global__ void __launch_bounds__(256) k_carry32(WalkArgs w, WalkArgs r) {
    extern __shared__ __align__(16) char smem[];
    float* phi = reinterpret_cast<float*>(smem);  // [2][N][N + 1]
    __shared__ __align__(16) float s_x[2][la::kMaxN][kCarryCols];
    const bool back = blockIdx.y == 1;
    const WalkArgs& a = back ? r : w;
    const int tid = threadIdx.x, N = (int)w.a.N, LD = N + 1, n = tid >> 1, c0 = (tid & 1) * 4, K = (int)w.plan.K;
    const int64_t P = w.a.P, ptiles = (P + kCarryCols - 1) / kCarryCols, p0 = blockIdx.x % ptiles * kCarryCols + c0, bh = blockIdx.x / ptiles;
    auto load = [&](int i) {
        const float* from = w.seg_phi + (bh * K + (back ? K - 1 - i : i)) * N * N;
        float* to = phi + (i & 1) * N * LD;
        for (int e = tid; e < N * N; e += 256)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(to + e / N * LD + e % N)), "l"(from + e) : "memory");
        copy_commit();
    };
    float x[4];
#pragma unroll
    for (int c = 0; c < 4; c++) x[c] = n < N && p0 + c < P && a.init ? a.init[(bh * N + n) * P + p0 + c] : 0.0f;
    load(0);
    for (int i = 0; i < K; i++) {
        float* at = a.seg_state + ((bh * K + (back ? K - 1 - i : i)) * N + n) * P + p0;
        float e[4] = {};
#pragma unroll
        for (int c = 0; c < 4; c++)
            if (n < N && p0 + c < P) {
                if (i + 1 < K) e[c] = at[c];
                at[c] = x[c];
            }
        if (i + 1 == K) break;
        if (n < N) *reinterpret_cast<float4*>(&s_x[i & 1][n][c0]) = make_float4(x[0], x[1], x[2], x[3]);
        copy_wait();
        __syncthreads();  // (and: the Phi before is used)
        if (i + 2 < K) load(i + 1);
        if (n < N) {
            const float* f = phi + (i & 1) * N * LD + (back ? n : n * LD);
            const int step = back ? LD : 1;
            float y[4] = {};
#pragma unroll 8
            for (int m = 0; m < N; m++) {
                const float p = f[m * step];
                const float4 z = at4(&s_x[i & 1][m][c0]);
                y[0] = fmaf(p, z.x, y[0]);
                y[1] = fmaf(p, z.y, y[1]);
                y[2] = fmaf(p, z.z, y[2]);
                y[3] = fmaf(p, z.w, y[3]);
            }
#pragma unroll
            for (int c = 0; c < 4; c++) x[c] = e[c] + y[c];
        }
    }
}

// ---------------------------------------------------------------- one chunk of one head
constexpr int C = kChunk;
constexpr int kPT = 64;  // value channels per pass
constexpr int kLdP = kPT + 4;

template <int NB> struct ChunkSmem {
    static constexpr int NP = NB * 16, LD = NP + 4;
    float q[C][LD], k[C][LD];
    float u[C][kLdP], dy[C][kLdP], x[C][kLdP];  // after the last pass: E in dy, F in x
    float H[NP][kLdP], R[NP][kLdP];
    Two c[C];
    float beta[C], a[C], b[C], db[C], col[8][C], red[8];
};

// Thread (ty, tx) of 16 x 16: rows 4 ty + r and columns tx + 16 n of the products with
// H, R, q, k; rows ty + 16 r and columns tx + 16 c of the 64 x 64 scores.
template <typename T, int NB> __global__ void __launch_bounds__(256) k_chunk(ChunkArgs w) {
    extern __shared__ __align__(16) char raw[];
    using Sm = ChunkSmem<NB>;
    Sm& s = *reinterpret_cast<Sm*>(raw);
    constexpr int NP = Sm::NP;
    const Args& a = w.a;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, lane = tid & 31, warp = tid >> 5;
    int64_t id = blockIdx.x;
    const int64_t h = id % a.H;
    id /= a.H;
    const int64_t chunk = id % w.chunks, b = id / w.chunks, rep = a.H / a.G, hq = h / rep;
    const int64_t t0 = chunk * C, len = row_length(a, b);
    const int nt = (int)min((int64_t)C, a.L - t0);
    const int nv = (int)max((int64_t)0, min((int64_t)nt, len - t0));

    const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + t0 * a.q.token + hq * a.N;
    const T* kp = static_cast<const T*>(a.k.p) + b * a.k.batch + t0 * a.k.token + hq * a.N;
#pragma unroll 8
    for (int u = 0; u < C * NP / 256; u++) {
        const int e = tid + 256 * u, t = e / NP, n = e % NP;
        const bool on = t < nv && n < a.N;
        s.q[t][n] = on ? ldf(qp + t * a.q.token + n) : 0.0f;
        s.k[t][n] = on ? ldf(kp + t * a.k.token + n) : 0.0f;
    }
    if (warp == 0) {
        float g[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int t = lane * 2 + e;
            g[e] = t < nv ? log_decay(a, b, t0 + t, h) * la::kLog2e : 0.0f;
            s.beta[t] = t < nv ? a.beta[(b * a.L + t0 + t) * a.H + h] : 0.0f;
        }
        Two c[2];
        la::warp_cumsum<2>(g, c);
        s.c[lane * 2] = c[0];
        s.c[lane * 2 + 1] = c[1];
    } else if (tid >= 64 && tid < 64 + C) {
        s.a[tid - 64] = s.b[tid - 64] = s.db[tid - 64] = 0.0f;
    }
    float through = 0.0f;
    float eu[4][4] = {}, fu[4][4] = {};                // dy . u, x . u
    float hd[4][NB] = {}, hx[4][NB] = {}, ru[4][NB] = {};  // H dy, H x, R u
    for (int64_t p0 = 0; p0 < a.P; p0 += kPT) {
        __syncthreads();
        const T* yp = static_cast<const T*>(a.dy.p) + b * a.dy.batch + t0 * a.dy.token + h * a.P + p0;
        const int64_t row0 = ((b * a.L + t0) * a.H + h) * a.P + p0;
#pragma unroll 2
        for (int u = 0; u < C / 8; u++) {
            const int t = warp + 8 * u;
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int p = lane + 32 * e;
                const bool on = t < nv && p0 + p < a.P;
                const float m = on ? w.miss[row0 + t * a.H * a.P + p] : 0.0f, x = on ? w.x[row0 + t * a.H * a.P + p] : 0.0f;
                s.u[t][p] = s.beta[t] * m;
                s.x[t][p] = x;
                s.dy[t][p] = on ? ldf(yp + t * a.dy.token + p) : 0.0f;
                sum = fmaf(m, x, sum);
            }
            sum = lane_sum<32>(sum);
            if (lane == 0) s.db[t] += sum;
        }
        const int64_t at = ((b * a.H + h) * w.chunks + chunk) * a.N * a.P + p0;
#pragma unroll 8
        for (int u = 0; u < NP * kPT / 256; u++) {
            const int e = tid + 256 * u, n = e / kPT, p = e % kPT;
            const bool on = nv > 0 && n < a.N && p0 + p < a.P;
            const float hv = on ? w.before[at + n * a.P + p] : 0.0f, rv = on ? w.after[at + n * a.P + p] : 0.0f;
            s.H[n][p] = hv;
            s.R[n][p] = rv;
            through = fmaf(hv, rv, through);
        }
        __syncthreads();
        for (int p = 0; p < kPT; p += 4) {
            float4 yv[4], xv[4], uv[4];
#pragma unroll
            for (int r = 0; r < 4; r++) yv[r] = at4(&s.dy[ty + 16 * r][p]), xv[r] = at4(&s.x[ty + 16 * r][p]), uv[r] = at4(&s.u[tx + 16 * r][p]);
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    eu[r][c] = fmaf(yv[r].x, uv[c].x, fmaf(yv[r].y, uv[c].y, fmaf(yv[r].z, uv[c].z, fmaf(yv[r].w, uv[c].w, eu[r][c]))));
                    fu[r][c] = fmaf(xv[r].x, uv[c].x, fmaf(xv[r].y, uv[c].y, fmaf(xv[r].z, uv[c].z, fmaf(xv[r].w, uv[c].w, fu[r][c]))));
                }
        }
        for (int p = 0; p < kPT; p += 4) {
            float4 yv[4], xv[4], uv[4];
#pragma unroll
            for (int r = 0; r < 4; r++) yv[r] = at4(&s.dy[4 * ty + r][p]), xv[r] = at4(&s.x[4 * ty + r][p]), uv[r] = at4(&s.u[4 * ty + r][p]);
#pragma unroll
            for (int n = 0; n < NB; n++) {
                const float4 hv = at4(&s.H[tx + 16 * n][p]), rv = at4(&s.R[tx + 16 * n][p]);
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    hd[r][n] = fmaf(yv[r].x, hv.x, fmaf(yv[r].y, hv.y, fmaf(yv[r].z, hv.z, fmaf(yv[r].w, hv.w, hd[r][n]))));
                    hx[r][n] = fmaf(xv[r].x, hv.x, fmaf(xv[r].y, hv.y, fmaf(xv[r].z, hv.z, fmaf(xv[r].w, hv.w, hx[r][n]))));
                    ru[r][n] = fmaf(uv[r].x, rv.x, fmaf(uv[r].y, rv.y, fmaf(uv[r].z, rv.z, fmaf(uv[r].w, rv.w, ru[r][n]))));
                }
            }
        }
    }
    float qk[4][4] = {}, kk[4][4] = {};
    for (int n = 0; n < NP; n += 4) {
        float4 qv[4], ki[4], kj[4];
#pragma unroll
        for (int r = 0; r < 4; r++) qv[r] = at4(&s.q[ty + 16 * r][n]), ki[r] = at4(&s.k[ty + 16 * r][n]), kj[r] = at4(&s.k[tx + 16 * r][n]);
#pragma unroll
        for (int r = 0; r < 4; r++)
#pragma unroll
            for (int c = 0; c < 4; c++) {
                qk[r][c] = fmaf(qv[r].x, kj[c].x, fmaf(qv[r].y, kj[c].y, fmaf(qv[r].z, kj[c].z, fmaf(qv[r].w, kj[c].w, qk[r][c]))));
                kk[r][c] = fmaf(ki[r].x, kj[c].x, fmaf(ki[r].y, kj[c].y, fmaf(ki[r].z, kj[c].z, fmaf(ki[r].w, kj[c].w, kk[r][c]))));
            }
    }
    __syncthreads();  // the last pass's tiles are read
    {
        float col[4] = {};
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int i = ty + 16 * r;
            float row = 0.0f;
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const int j = tx + 16 * c;
                const float m = j <= i ? la::ex2(two_diff(s.c[i], s.c[j])) : 0.0f;
                const float e = a.scale * m * eu[r][c], f = j < i ? -s.beta[i] * m * fu[r][c] : 0.0f;
                s.dy[i][j] = e;
                s.x[i][j] = f;
                const float x = j < i ? fmaf(e, qk[r][c], f * kk[r][c]) : 0.0f;
                row += x;
                col[c] += x;
            }
            row = lane_sum<16>(row);
            if (tx == 0) s.b[i] -= row;
        }
#pragma unroll
        for (int c = 0; c < 4; c++) {
            col[c] += __shfl_xor_sync(kFull, col[c], 16);
            if (lane < 16) s.col[warp][tx + 16 * c] = col[c];
        }
    }
    __syncthreads();
    if (tid < C) {
        float x = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; u++) x += s.col[u][tid];
        s.b[tid] += x;
    }
    __syncthreads();
    const Two cl = s.c[C - 1];
    float dq[4][NB], dk[4][NB];
#pragma unroll
    for (int r = 0; r < 4; r++) {
        const int i = 4 * ty + r;
        const float up = la::ex2(s.c[i].h + s.c[i].l), down = la::ex2(two_diff(cl, s.c[i])), beta = s.beta[i];
        float ai = 0.0f, bi = 0.0f;
#pragma unroll
        for (int n = 0; n < NB; n++) {
            const int m = tx + 16 * n;
            dq[r][n] = a.scale * up * hd[r][n];
            const float in = -beta * up * hx[r][n], to = down * ru[r][n];
            dk[r][n] = in + to;
            ai = fmaf(s.q[i][m], dq[r][n], fmaf(s.k[i][m], in, ai));
            bi = fmaf(s.k[i][m], to, bi);
        }
        ai = lane_sum<16>(ai);
        bi = lane_sum<16>(bi);
        if (tx == 0) {
            s.a[i] = ai;
            s.b[i] += bi;
        }
    }
    for (int j = 0; j < C; j += 4) {  // E k, F k: rows i of E, F
        float4 e[4], f[4];
#pragma unroll
        for (int r = 0; r < 4; r++) e[r] = at4(&s.dy[4 * ty + r][j]), f[r] = at4(&s.x[4 * ty + r][j]);
#pragma unroll
        for (int n = 0; n < NB; n++) {
            const int m = tx + 16 * n;
            const float k0 = s.k[j][m], k1 = s.k[j + 1][m], k2 = s.k[j + 2][m], k3 = s.k[j + 3][m];
#pragma unroll
            for (int r = 0; r < 4; r++) {
                dq[r][n] = fmaf(e[r].x, k0, fmaf(e[r].y, k1, fmaf(e[r].z, k2, fmaf(e[r].w, k3, dq[r][n]))));
                dk[r][n] = fmaf(f[r].x, k0, fmaf(f[r].y, k1, fmaf(f[r].z, k2, fmaf(f[r].w, k3, dk[r][n]))));
            }
        }
    }
#pragma unroll 2
    for (int i = 0; i < C; i++) {  // E^T q, F^T k: columns
        const float4 e = at4(&s.dy[i][4 * ty]), f = at4(&s.x[i][4 * ty]);
        const float es[4] = {e.x, e.y, e.z, e.w}, fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int n = 0; n < NB; n++) {
            const float q = s.q[i][tx + 16 * n], k = s.k[i][tx + 16 * n];
#pragma unroll
            for (int r = 0; r < 4; r++) dk[r][n] = fmaf(es[r], q, fmaf(fs[r], k, dk[r][n]));
        }
    }
#pragma unroll
    for (int r = 0; r < 4; r++) {
        const int t = 4 * ty + r;
        if (t >= nt) continue;
#pragma unroll
        for (int n = 0; n < NB; n++) {
            const int c = tx + 16 * n;
            if (c >= a.N) continue;
            const int64_t at = ((b * a.L + t0 + t) * a.G + hq) * a.N + c;
            const float x = t < nv ? dq[r][n] : 0.0f, z = t < nv ? dk[r][n] : 0.0f;
            if (rep > 1) {
                const int64_t part = (h % rep) * a.Bsz * a.L * a.G * a.N + at;
                w.dq_part[part] = x;
                w.dk_part[part] = z;
            } else {
                st(static_cast<T*>(w.dq) + at, x);
                st(static_cast<T*>(w.dk) + at, z);
            }
        }
    }
    through = lane_sum<32>(through);
    if (lane == 0) s.red[warp] = through;
    __syncthreads();
    if (warp == 0) {
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; u++) sum += s.red[u];
        sum *= la::ex2(cl.h + cl.l);
        const int t = 2 * lane;
        const float a0 = s.a[t], a1 = s.a[t + 1], b0 = s.b[t], b1 = s.b[t + 1];
        float A = a0 + a1, B = b0 + b1;  // suffix of a, prefix of b over lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_down_sync(kFull, A, o), y = __shfl_up_sync(kFull, B, o);
            if (lane + o < 32) A += x;
            if (lane >= o) B += y;
        }
        const float Bx = __shfl_up_sync(kFull, B, 1), Ax = __shfl_down_sync(kFull, A, 1);
        const float pre = lane > 0 ? Bx : 0.0f, suf = lane < 31 ? Ax : 0.0f;
        const float g[2] = {(a0 + a1 + suf) + pre + sum, (a1 + suf) + (pre + b0) + sum};
#pragma unroll
        for (int e = 0; e < 2; e++)
            if (t + e < nt) {
                const int64_t at = (b * a.L + t0 + t + e) * a.H + h;
                if (w.dg) w.dg[at] = t + e < nv ? g[e] : 0.0f;
                w.dbeta[at] = t + e < nv ? s.db[t + e] : 0.0f;
            }
    }
}

enum Launch { kOne, kBoth, kSums };
template <typename T, int LN> cudaError_t walk_go(Launch what, const WalkArgs& w, const WalkArgs* back, cudaStream_t st) {
    constexpr int y = 2 * sizeof(WalkStage<LN, kWalkY>), sum = 2 * sizeof(WalkStage<LN, kWalkSum>);
    const int64_t rows = w.a.H * w.a.Bsz * w.plan.K, wide = ceil_div(w.a.P, 64 / LN), deep = ceil_div(w.a.N, 64 / LN);
    const unsigned grid = (unsigned)(wide * rows);
    if (what == kOne) (grid > 4 * kSms ? k_walk<T, LN, 6> : k_walk<T, LN, 1>)<<<grid, 64, y, st>>>(w);
    else if (what == kBoth) (2 * (int64_t)grid > 4 * kSms ? k_walks<T, LN, 6> : k_walks<T, LN, 1>)<<<dim3(grid, 2), 64, y, st>>>(w, *back);
    else k_sums<T, LN><<<dim3((unsigned)((wide > deep ? wide : deep) * rows), back ? 3 : 2), 64, back ? y : sum, st>>>(w, back ? *back : w);
    return cudaGetLastError();
}
template <typename T> cudaError_t walk_io(Launch what, const WalkArgs& w, const WalkArgs* back, cudaStream_t st) {
    switch (walk_lanes(w.a.N)) {
        case 1: return walk_go<T, 1>(what, w, back, st);
        case 2: return walk_go<T, 2>(what, w, back, st);
        case 4: return walk_go<T, 4>(what, w, back, st);
        default: return walk_go<T, 8>(what, w, back, st);
    }
}

template <typename T, int NB> cudaError_t chunk_n(const ChunkArgs& c, cudaStream_t st) {
    const int bytes = (int)sizeof(ChunkSmem<NB>);
    const cudaError_t e = la::allow_smem<k_chunk<T, NB>>(bytes);
    if (e != cudaSuccess) return e;
    k_chunk<T, NB><<<(unsigned)(c.a.Bsz * c.chunks * c.a.H), 256, bytes, st>>>(c);
    return cudaGetLastError();
}
template <typename T> cudaError_t chunk_io(const ChunkArgs& c, cudaStream_t st) {
    if (c.a.N <= 32) return chunk_n<T, 2>(c, st);
    if (c.a.N <= 64) return chunk_n<T, 4>(c, st);
    return chunk_n<T, 8>(c, st);
}

// Whether q, k, v and dy are f32 and every run of four values is whole and aligned.
bool fours(const Args& a) {
    if (a.dtype != 0) return false;
    for (const In* x : {&a.q, &a.k, &a.v, &a.dy})
        if (reinterpret_cast<uintptr_t>(x->p) % 16 != 0 || x->token % 4 != 0 || x->batch % 4 != 0) return false;
    return a.N % 4 == 0 && a.P % 4 == 0;
}

}  // namespace

static cudaError_t go(Launch what, WalkArgs w, const WalkArgs* back, cudaStream_t st) {
    w.vec = fours(w.a);
    WalkArgs r;
    if (back) {
        r = *back;
        r.vec = w.vec;
        back = &r;
    }
    if (w.a.dtype == 0) return walk_io<float>(what, w, back, st);
    if (w.a.dtype == 1) return walk_io<__half>(what, w, back, st);
    return walk_io<__nv_bfloat16>(what, w, back, st);
}
cudaError_t launch_pairs(const Args& a, Pairs* pairs, cudaStream_t st) {
    const int64_t tiles = ceil_div(a.L, kWalkT);
    const unsigned grid = (unsigned)(a.Bsz * a.H * tiles);
    if (a.dtype == 0) k_pairs<float><<<grid, 128, 0, st>>>(a, pairs, tiles);
    else if (a.dtype == 1) k_pairs<__half><<<grid, 128, 0, st>>>(a, pairs, tiles);
    else k_pairs<__nv_bfloat16><<<grid, 128, 0, st>>>(a, pairs, tiles);
    return cudaGetLastError();
}
cudaError_t launch_walk(const WalkArgs& w, cudaStream_t st) { return go(kOne, w, nullptr, st); }
cudaError_t launch_walks(const WalkArgs& keep, const WalkArgs& back, cudaStream_t st) { return go(kBoth, keep, &back, st); }
cudaError_t launch_segments(const WalkArgs& w, const WalkArgs* back, cudaStream_t st) {
    cudaError_t e = go(kSums, w, back, st);
    if (e != cudaSuccess) return e;
    e = la::allow_smem<k_carry32>(2 * la::kMaxN * (la::kMaxN + 1) * 4);
    if (e != cudaSuccess) return e;
    const int N = (int)w.a.N;
    k_carry32<<<dim3((unsigned)(ceil_div(w.a.P, kCarryCols) * w.a.Bsz * w.a.H), back ? 2 : 1), 256, 2 * N * (N + 1) * 4, st>>>(w, back ? *back : w);
    return cudaGetLastError();
}

// Costs in tiles walked by a block alone on its SM.  Blocks beside it, measured: two take 1.05 to 1.18 of its time, three 1.34 to
// 1.48, four 1.4 to 1.8, five 1.9 to 2.1, six 1.9 to 2.3, and further ones begin another round.  A segment's carry is most of a tile's time, two launches two.
WalkPlan walk_plan(int64_t heads, int64_t N, int64_t P, int64_t L, bool backward) {
    const int64_t pt = 64 / walk_lanes(N), wide = ceil_div(P, pt), deep = ceil_div(N, pt), tiles = ceil_div(L, kWalkT), chunk = kChunk / kWalkT;
    const int64_t both = backward ? 2 : 1;
    auto rounds = [](int64_t blocks) {
        constexpr double beside[6] = {0.0, 1.0, 1.1, 1.4, 1.65, 2.0};
        const int64_t n = ceil_div(blocks, kSms);
        return 2.2 * (double)(n / 6) + beside[n % 6];
    };
    WalkPlan best = {1, tiles};
    double least = rounds(heads * wide * both) * tiles;
    for (int64_t K = 2; K <= 64 && 2 * K * chunk <= tiles; K++) {
        const int64_t seg = ceil_div(ceil_div(tiles, K), chunk) * chunk;
        if (ceil_div(tiles, seg) != K) continue;
        const int64_t sums = heads * (wide * both * (K - 1) + deep * (backward ? K : K - 1));
        const double cost = (rounds(sums) + rounds(heads * wide * both * K)) * seg + 0.8 * K + 2;
        if (cost < 0.9 * least) {
            least = cost;
            best = {K, seg};
        }
    }
    return best;
}

cudaError_t launch_chunks(const ChunkArgs& c, cudaStream_t st) {
    if (c.a.dtype == 0) return chunk_io<float>(c, st);
    if (c.a.dtype == 1) return chunk_io<__half>(c, st);
    return chunk_io<__nv_bfloat16>(c, st);
}

}  // namespace gdr
}  // namespace ss
