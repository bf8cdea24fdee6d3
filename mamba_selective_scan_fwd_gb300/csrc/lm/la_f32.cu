// Linear attention on the FP32 units: every io type, any N <= 128, P and
// strides.  f32 inputs run here, and 16-bit inputs that the tensor-core path's
// 16-byte rules exclude.
//
// The forward's walk is the recurrence itself, token by token with the state in
// registers: 3 N P operations per token and head, fewer than any chunked form takes
// without matrix units.  In a
// tile of at most 16 tokens whose decay stays at e^-4 or weaker (kSlowTile) the state at
// its start stays as it is and what the tile adds is summed apart, in units of the
// decay since the start: the same operations, and the state is rounded once a tile
// instead of twice a token, which a long memory adds up (2 x 3294 tokens, f32:
// 1.4e-6 -> 2e-7 of f64).  Under a stronger decay the tokens enter one by one (their
// decays: Decay in la_dev.cuh).  The backward works on chunks of 64 tokens from the states at their
// borders, which are the carried sums of the chunks.
//
// Measured, f32: 2 x 1000 tokens, 24 heads, N = P = 64: sums 20 us, carries 6, walk 47
// (57 % of the issue slots, shared memory 41 %; without the slow-decay form 5 us less);
// uncut 204.  Backward of 777 tokens, 16 heads, N 32, P 64: sums 11 us, carries 6, chunks
// 32, parts 4.
#include <type_traits>

#include "../simd.cuh"
#include "la_dev.cuh"

namespace ss {
namespace la {
namespace {

constexpr float kSlowTile = -4.0f;  // every c of the tile between it and its opposite: e^-c stays between 1 / 55 and 55

__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// Four adjacent values, of which `left` exist; vec: they exist together and are aligned.
template <typename T> __device__ __forceinline__ float4 fetch4(const T* p, int64_t left, bool vec) {
    float x[4] = {};
    if (vec) {
        if (left > 0) {
            if constexpr (sizeof(T) == 4) return at4(p);
            union {
                uint2 m;
                T t[4];
            } u;
            u.m = *reinterpret_cast<const uint2*>(p);
#pragma unroll
            for (int e = 0; e < 4; e++) x[e] = ldf(&u.t[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = e < left ? ldf(p + e) : 0.0f;
    }
    return make_float4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ float2 decayed2(Decay d, float2 x) {
    return d.weak ? fma2(splat2(d.by), x, x) : mul2(splat2(d.by), x);
}

// End states of the segments, each walked from zero.  One block: kWalkP value
// channels of one head, one segment, in tiles of TT tokens:
//   forward   X <- e^{cl} X + k^T (e^{cl - c} v)
//   reverse   X <- e^{cl} X + q^T (scale e^c dy), tiles last to first
// with c the cumulative log decay in the tile and cl its end.  Thread (ty, tx) of
// 16 x 16: RN rows and four columns of X, read 16 bytes of k and v a token.
template <typename T, int RN>
__global__ void __launch_bounds__(256, RN == 8 ? 2 : 3) k_sum32(WalkArgs w) {
    constexpr int NP = RN * 16, TT = RN == 8 ? 16 : 32;
    constexpr int EK = TT * NP / 1024 < 1 ? 1 : TT * NP / 1024, EV = TT * kWalkP / 1024;  // runs of 4 values a thread loads
    __shared__ __align__(16) float s_k[2][TT][NP], s_v[2][TT][kWalkP];
    __shared__ float2 s_w[2][TT];  // (a token's weight, twice)
    __shared__ float s_all[2];
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tx = tid & 15, ty = tid >> 4;
    const int64_t ptiles = (a.P + kWalkP - 1) / kWalkP, segs = w.dirs == 1 ? w.plan.K - 1 : w.plan.K;
    int64_t id = blockIdx.x;
    const int64_t p0 = (id % ptiles) * kWalkP;
    id /= ptiles;
    const int64_t h = id % a.H;
    id /= a.H;
    const int64_t seg = id % segs;
    id /= segs;
    const int64_t b = id % a.Bsz;
    const bool rev = id / a.Bsz != 0;
    const int64_t hq = h / (a.H / a.G), at = ((rev ? a.Bsz * a.H : 0) + b * a.H + h) * w.plan.K + seg;
    const int64_t t_begin = seg * w.plan.seg, t_end = min(a.L, t_begin + w.plan.seg), len = row_length(a, b);
    const In &kin = rev ? a.q : a.k, &vin = rev ? a.dy : a.v;
    const T* kp = static_cast<const T*>(kin.p) + b * kin.batch + hq * a.N;
    const T* vp = static_cast<const T*>(vin.p) + b * vin.batch + h * a.P + p0;
    const int tiles = (int)((t_end - t_begin + TT - 1) / TT), N = (int)a.N, pleft = (int)(a.P - p0);

    float4 rk[EK], rv[EV];
    float rg = 0.0f;
    auto fetch = [&](int i) {
        const int64_t t0 = t_begin + (int64_t)(rev ? tiles - 1 - i : i) * TT;
        const int nv = (int)max((int64_t)0, min((int64_t)TT, min(len, t_end) - t0));
        const T *k0 = kp + t0 * kin.token, *v0 = vp + t0 * vin.token;
#pragma unroll
        for (int e = 0; e < EK; e++) {
            const int x = tid + 256 * e, t = x / (NP / 4), n = x % (NP / 4) * 4;
            rk[e] = fetch4(k0 + t * kin.token + n, t < nv ? N - n : 0, w.vec);
        }
#pragma unroll
        for (int e = 0; e < EV; e++) {
            const int x = tid + 256 * e, t = x / (kWalkP / 4), c = x % (kWalkP / 4) * 4;
            rv[e] = fetch4(v0 + t * vin.token + c, t < nv ? pleft - c : 0, w.vec);
        }
        if (warp == 0) rg = lane < nv ? log_decay(a, b, t0 + lane, h) : 0.0f;
    };
    fetch(0);
    float2 S[RN / 2][4] = {};  // pairs of rows
    float total = 0.0f;
    for (int i = 0; i < tiles; i++) {
        const int s = i & 1;
#pragma unroll
        for (int e = 0; e < EK; e++)
            if (TT * NP >= 1024 || tid < TT * NP / 4) reinterpret_cast<float4*>(s_k[s])[tid + 256 * e] = rk[e];
#pragma unroll
        for (int e = 0; e < EV; e++) reinterpret_cast<float4*>(s_v[s])[tid + 256 * e] = rv[e];
        if (warp == 0) {
            const float x[1] = {rg};
            Two c[1];
            warp_cumsum<1>(x, c);
            const Two cl = {__shfl_sync(kFull, c[0].h, 31), __shfl_sync(kFull, c[0].l, 31)};
            if (lane < TT) s_w[s][lane] = splat2(rev ? a.scale * expf(c[0].h) * (1.0f + c[0].l) : expf(two_diff(cl, c[0])));
            if (lane == 0) s_all[s] = cl.h + cl.l;
        }
        __syncthreads();
        if (i + 1 < tiles) fetch(i + 1);
        float2 X[RN / 2][4] = {};
#pragma unroll 8
        for (int t = 0; t < TT; t++) {
            const float4 v = at4(&s_v[s][t][4 * tx]);
            const float2 wt = s_w[s][t], vs[4] = {splat2(v.x), splat2(v.y), splat2(v.z), splat2(v.w)};
#pragma unroll
            for (int r = 0; r < RN / 2; r++) {
                const float2 k = mul2(wt, *reinterpret_cast<const float2*>(&s_k[s][t][RN * ty + 2 * r]));
#pragma unroll
                for (int c = 0; c < 4; c++) X[r][c] = fma2(k, vs[c], X[r][c]);
            }
        }
        const float all = s_all[s];
        const Decay d = decay_of(all);
        total += all;
#pragma unroll
        for (int r = 0; r < RN / 2; r++)
#pragma unroll
            for (int c = 0; c < 4; c++) S[r][c] = add2(decayed2(d, S[r][c]), X[r][c]);
    }
    float* to = w.seg_state + at * a.N * a.P + p0 + 4 * tx;
#pragma unroll
    for (int r = 0; r < RN; r++) {
        const int n = RN * ty + r;
        if (n >= N) continue;
        const float4 x = r & 1 ? make_float4(S[r / 2][0].y, S[r / 2][1].y, S[r / 2][2].y, S[r / 2][3].y)
                               : make_float4(S[r / 2][0].x, S[r / 2][1].x, S[r / 2][2].x, S[r / 2][3].x);
        float* row = to + n * a.P;
        if (w.vec) {
            if (4 * tx < pleft) *reinterpret_cast<float4*>(row) = x;
        } else {
            const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int c = 0; c < 4; c++)
                if (4 * tx + c < pleft) row[c] = y[c];
        }
    }
    if (tid == 0 && p0 == 0) w.seg_decay[at] = total;
}

// y.  One block: kWalkP value channels of one head, one segment of tokens.  Lane = two
// value channels 32 apart, warp = NR of the padded N state rows, in pairs.  The
// rows' k and q are broadcasts from shared memory, which is what bounds it: two
// channels a lane halve them.
// The next TT tokens are loaded into registers while these are computed.
template <typename T, int NR>
__global__ void __launch_bounds__(256, NR == 16 ? 2 : 3) k_walk32(WalkArgs w) {
    constexpr int NP = NR * 8, TT = NR == 16 ? kWalkT / 2 : kWalkT;
    constexpr int EK = TT * NP / 1024 < 1 ? 1 : TT * NP / 1024, EV = TT * kWalkP / 1024 < 1 ? 1 : TT * kWalkP / 1024;  // runs of 4 values a thread loads
    __shared__ __align__(16) float s_k[TT][NP], s_q[TT][NP], s_v[TT][kWalkP];
    __shared__ float s_a[TT], s_down[TT], s_up[TT], s_all;
    __shared__ uint32_t s_weak;  // bit t: token t's decay is weak
    __shared__ bool s_slow;
    __shared__ float s_y[8][TT][kWalkP];
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t ptiles = (a.P + kWalkP - 1) / kWalkP;
    int64_t id = blockIdx.x;
    const int64_t p0 = (id % ptiles) * kWalkP;
    id /= ptiles;
    const int64_t h = id % a.H;
    id /= a.H;
    const int64_t seg = id % w.plan.K, b = id / w.plan.K;
    const int64_t hq = h / (a.H / a.G), bh = b * a.H + h;
    const int64_t t_begin = seg * w.plan.seg, t_end = min(a.L, t_begin + w.plan.seg);
    const int64_t len = row_length(a, b);
    const int n0 = warp * NR, N = (int)a.N, pleft = (int)(a.P - p0);
    const int64_t NPel = a.N * a.P;
    const T* kp = static_cast<const T*>(a.k.p) + b * a.k.batch + hq * a.N;
    const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + hq * a.N;
    const T* vp = static_cast<const T*>(a.v.p) + b * a.v.batch + h * a.P + p0;
    const WalkDir& dir = w.dir[0];

    float2 S[2][NR / 2];  // [channel][pair of rows]
    const float* init = w.plan.K > 1 ? w.seg_state + (bh * w.plan.K + seg) * NPel : (dir.init ? dir.init + bh * NPel : nullptr);
#pragma unroll
    for (int c = 0; c < 2; c++) {
        const int64_t p = p0 + lane + 32 * c;
        auto from = [&](int n) { return init && n < a.N && p < a.P ? init[n * a.P + p] : 0.0f; };
#pragma unroll
        for (int r = 0; r < NR / 2; r++) S[c][r] = make_float2(from(n0 + 2 * r), from(n0 + 2 * r + 1));
    }

    const int64_t tiles = (t_end - t_begin + TT - 1) / TT;
    auto valid = [&](int64_t t0) { return (int)max((int64_t)0, min((int64_t)TT, min(len, t_end) - t0)); };  // tokens that count
    float4 rk[EK], rq[EK], rv[EV];
    float rg = 0.0f;
    auto fetch = [&](int64_t i) {
        const int64_t t0 = t_begin + i * TT;
        const int nv = valid(t0);
        const T *k0 = kp + t0 * a.k.token, *q0 = qp + t0 * a.q.token, *v0 = vp + t0 * a.v.token;
#pragma unroll
        for (int e = 0; e < EK; e++) {
            const int x = tid + 256 * e, t = x / (NP / 4), n = x % (NP / 4) * 4, left = t < nv ? N - n : 0;
            rk[e] = fetch4(k0 + t * a.k.token + n, left, w.vec);
            rq[e] = fetch4(q0 + t * a.q.token + n, left, w.vec);
        }
#pragma unroll
        for (int e = 0; e < EV; e++) {
            const int x = tid + 256 * e, t = x / (kWalkP / 4), c = x % (kWalkP / 4) * 4;
            rv[e] = fetch4(v0 + t * a.v.token + c, t < nv ? pleft - c : 0, w.vec);
        }
        if (tid < TT) rg = tid < nv ? log_decay(a, b, t0 + tid, h) : 0.0f;
    };
    fetch(0);
    for (int64_t i = 0; i < tiles; i++) {
        const int64_t t0 = t_begin + i * TT;
        const int nv = valid(t0);
        __syncthreads();
#pragma unroll
        for (int e = 0; e < EK; e++)
            if (TT * NP >= 1024 || tid < TT * NP / 4) {
                reinterpret_cast<float4*>(s_k)[tid + 256 * e] = rk[e];
                reinterpret_cast<float4*>(s_q)[tid + 256 * e] = rq[e];
            }
#pragma unroll
        for (int e = 0; e < EV; e++)
            if (TT * kWalkP >= 1024 || tid < TT * kWalkP / 4) reinterpret_cast<float4*>(s_v)[tid + 256 * e] = rv[e];
        if (warp == 0) {  // the tile's decays
            const float x[1] = {lane < TT ? rg : 0.0f};
            Two c[1];
            warp_cumsum<1>(x, c);
            const bool slow = __all_sync(kFull, c[0].h >= kSlowTile && c[0].h <= -kSlowTile);  // (NaN: no)
            if (lane == 31) {
                s_all = c[0].h + c[0].l;
                s_slow = slow;
            }
            const Decay d = decay_of(x[0]);
            const uint32_t weak = __ballot_sync(kFull, d.weak);
            if (lane == 0) s_weak = weak;
            if (lane < TT) {
                s_a[lane] = d.by;
                s_down[lane] = expf(-c[0].h) * (1.0f - c[0].l);
                s_up[lane] = expf(c[0].h) * (1.0f + c[0].l);
            }
        }
        __syncthreads();
        if (i + 1 < tiles) fetch(i + 1);
        const float all = s_all;
        const bool slow = s_slow;
        const uint32_t weak = s_weak;
        // SLOW: S = S0 + A in units of e^c: S0 stays, A takes what the tile adds
        auto tokens = [&](auto which) {
            constexpr bool SLOW = decltype(which)::value;
            float2 A[2][NR / 2] = {};
            auto token = [&](int t, auto how) {
                constexpr bool WEAK = decltype(how)::value;
                const float d = SLOW ? s_down[t] : 1.0f;
                const float2 av = splat2(s_a[t]), v[2] = {splat2(s_v[t][lane] * d), splat2(s_v[t][lane + 32] * d)};
                float2 acc[2][2] = {};
#pragma unroll
                for (int r = 0; r < NR / 2; r += 2) {
                    const float4 kk = at4(&s_k[t][n0 + 2 * r]), qq = at4(&s_q[t][n0 + 2 * r]);
                    const float2 kr[2] = {make_float2(kk.x, kk.y), make_float2(kk.z, kk.w)};
                    const float2 qr[2] = {make_float2(qq.x, qq.y), make_float2(qq.z, qq.w)};
#pragma unroll
                    for (int c = 0; c < 2; c++)
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            float2 &x = S[c][r + u], &y = A[c][r + u];
                            if (SLOW) y = fma2(kr[u], v[c], y);
                            else x = fma2(kr[u], v[c], WEAK ? fma2(av, x, x) : mul2(av, x));
                            acc[c][u] = fma2(qr[u], SLOW ? add2(x, y) : x, acc[c][u]);
                        }
                }
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    const float2 s = add2(acc[c][0], acc[c][1]);
                    s_y[warp][t][lane + 32 * c] = s.x + s.y;
                }
            };
#pragma unroll 2
            for (int t = 0; t < nv; t++) {
                if (SLOW || (weak >> t & 1)) token(t, std::true_type{});
                else token(t, std::false_type{});
            }
            if (SLOW) {
                const Decay d = decay_of(all);
#pragma unroll
                for (int c = 0; c < 2; c++)
#pragma unroll
                    for (int r = 0; r < NR / 2; r++) S[c][r] = decayed2(d, add2(S[c][r], A[c][r]));
            }
        };
        if (slow) tokens(std::true_type{});
        else tokens(std::false_type{});
        __syncthreads();
        T* yp = static_cast<T*>(w.y) + ((b * a.L + t0) * a.H + h) * a.P + p0;
        const int nt = (int)min((int64_t)TT, t_end - t0);
#pragma unroll
        for (int u = 0; u < TT * kWalkP / 256; u++) {
            const int e = tid + 256 * u, t = e / kWalkP, c = e % kWalkP;
            if (t < nt && c < pleft) {
                float y = 0.0f;
                if (t < nv) {
#pragma unroll
                    for (int o = 0; o < 8; o++) y += s_y[o][t][c];
                }
                st(yp + t * a.H * a.P + c, a.scale * (slow ? s_up[t] * y : y));
            }
        }
    }
    if (dir.last && seg == w.plan.K - 1) {
        float* dst = dir.last + bh * NPel;
#pragma unroll
        for (int c = 0; c < 2; c++) {
            const int64_t p = p0 + lane + 32 * c;
#pragma unroll
            for (int r = 0; r < NR / 2; r++) {
                if (n0 + 2 * r < a.N && p < a.P) dst[(n0 + 2 * r) * a.P + p] = S[c][r].x;
                if (n0 + 2 * r + 1 < a.N && p < a.P) dst[(n0 + 2 * r + 1) * a.P + p] = S[c][r].y;
            }
        }
    }
}

// seg_state: end state of each segment walked from zero -> the state each
// segment starts from.  One thread per state element; 16 segments' states are on
// their way before the first is folded in (one memory wait per 16).
__global__ void __launch_bounds__(256) k_carry32(WalkArgs w, int64_t first) {
    constexpr int U = 16;
    const int64_t K = w.plan.K, BH = w.a.Bsz * w.a.H, NP = w.a.N * w.a.P;
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, unit = first + blockIdx.y;
    if (x >= NP) return;
    const bool rev = unit >= BH;
    const float* init = w.dir[rev].init;
    float S = init ? init[(unit - (rev ? BH : 0)) * NP + x] : 0.0f;
    const int64_t sums = w.dirs == 1 ? K - 1 : K;
    for (int64_t i0 = 0; i0 < K; i0 += U) {
        float own[U], d[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t i = i0 + u, s = unit * K + (rev ? K - 1 - i : i);
            own[u] = d[u] = 0.0f;
            if (i < sums) {
                own[u] = w.seg_state[s * NP + x];
                d[u] = expf(w.seg_decay[s]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t i = i0 + u, s = unit * K + (rev ? K - 1 - i : i);
            if (i < K) w.seg_state[s * NP + x] = S;
            if (i < sums) S = fmaf(d[u], S, own[u]);
        }
    }
    float* last = w.dir[rev].last;
    if (w.dirs == 2 && last) last[(unit - (rev ? BH : 0)) * NP + x] = S;
}

// ---------------------------------------------------------------- backward, one chunk of one group of heads
constexpr int kPT = 64;  // value channels per pass
constexpr int kLdP = kPT + 4;

template <int NB> struct Smem32 {
    static constexpr int NP = NB * 16, LD = NP + 4;
    float q[kChunk32][LD], k[kChunk32][LD];
    float v[kChunk32][kLdP], dy[kChunk32][kLdP];
    float E[kChunk32][kLdP], S[kChunk32][kLdP];  // decayed dy v^T and q k^T (rows i, columns j <= i)
    float H[NP][kLdP], R[NP][kLdP];
    Two c[kChunk32];
    float a[kChunk32], b[kChunk32], col[8][kChunk32], red[8];
};

// acc (4 adjacent values) += x z
__device__ __forceinline__ void fma4(float2 (&acc)[2], float x, float4 z) {
    acc[0] = fma2(splat2(x), make_float2(z.x, z.y), acc[0]);
    acc[1] = fma2(splat2(x), make_float2(z.z, z.w), acc[1]);
}
// acc (two halves of a sum) += x . z
__device__ __forceinline__ void dot4(float2& acc, float4 x, float4 z) {
    acc = fma2(make_float2(x.x, x.y), make_float2(z.x, z.y), acc);
    acc = fma2(make_float2(x.z, x.w), make_float2(z.z, z.w), acc);
}

// Thread (ty, tx) of 16 x 16 holds four rows and some columns of every product:
// rows and columns 16 apart where a product runs over the rows' own columns,
// adjacent ones where that makes a shared-memory read of 16 bytes.  Bound by the
// latencies of one block's steps: 208 blocks on 152 SMs at 777 tokens x 16 heads, a
// third of the issue slots used.  With c_i the cumulative log decay inside the chunk, cl its
// end, H the state before and R the adjoint after the chunk (all per head):
//   m_ij = scale e^{c_i - c_j} (j <= i),  E = m o (dy v^T),  S = m o (q k^T),  W = E o (q k^T)
//   dq = E k + scale e^{c} (dy H^T),  dk = E^T q + e^{cl - c} (v R^T),  dv = S^T dy + e^{cl - c} (k R)
//   dg_t = sum_{i >= t} a_i + sum_{j < t} (b_j + col_j - row_j) + e^{cl} <R, H>
// with a_i, b_j the inter-chunk parts of q.dq and k.dk and row, col the sums
// of W below the diagonal: col_j - row_j telescopes to the pairs that span t.
template <typename T, int NB>
__global__ void __launch_bounds__(256) k_bwd32(BwdArgs w) {
    extern __shared__ __align__(16) char raw[];
    using Sm = Smem32<NB>;
    Sm& s = *reinterpret_cast<Sm*>(raw);
    constexpr int C = kChunk32, NP = Sm::NP;
    const Args& a = w.a;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, lane = tid & 31, warp = tid >> 5;
    int64_t id = blockIdx.x;
    const int64_t split = id % w.splits;
    id /= w.splits;
    const int64_t gq = id % a.G;
    id /= a.G;
    const int64_t chunk = id % w.chunks, b = id / w.chunks;
    const int64_t t0 = chunk * C;
    const int64_t len = row_length(a, b);
    const int nt = (int)min((int64_t)C, a.L - t0);
    const int nv = (int)max((int64_t)0, min((int64_t)nt, len - t0));
    const int nc = (nv + 3) & ~3;  // sums over tokens end here: what follows is zero
    const int64_t rep = a.H / a.G;
    const int64_t h_lo = gq * rep + rep * split / w.splits, h_hi = gq * rep + rep * (split + 1) / w.splits;

    const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + t0 * a.q.token + gq * a.N;
    const T* kp = static_cast<const T*>(a.k.p) + b * a.k.batch + t0 * a.k.token + gq * a.N;
#pragma unroll 8
    for (int u = 0; u < C * NP / 256; u++) {
        const int e = tid + 256 * u, t = e / NP, n = e % NP;
        const bool on = t < nv && n < a.N;
        s.q[t][n] = on ? ldf(qp + t * a.q.token + n) : 0.0f;
        s.k[t][n] = on ? ldf(kp + t * a.k.token + n) : 0.0f;
    }
    float dq[4][NB] = {};
    float2 dk[2][NB] = {};  // pairs of rows

    for (int64_t h = h_lo; h < h_hi; h++) {
        __syncthreads();
        if (warp == 0) {
            float x[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int t = lane * 2 + e;
                x[e] = t < nv ? log_decay(a, b, t0 + t, h) * kLog2e : 0.0f;
            }
            Two c[2];
            warp_cumsum<2>(x, c);
            s.c[lane * 2] = c[0];
            s.c[lane * 2 + 1] = c[1];
        } else if (tid >= 64 && tid < 64 + C) {
            s.a[tid - 64] = s.b[tid - 64] = 0.0f;
        }
        float through = 0.0f;
        for (int64_t p0 = 0; p0 < a.P; p0 += kPT) {
            __syncthreads();
            const T* vp = static_cast<const T*>(a.v.p) + b * a.v.batch + t0 * a.v.token + h * a.P + p0;
            const T* yp = static_cast<const T*>(a.dy.p) + b * a.dy.batch + t0 * a.dy.token + h * a.P + p0;
#pragma unroll
            for (int u = 0; u < C * kPT / 256; u++) {
                const int e = tid + 256 * u, t = e / kPT, p = e % kPT;
                const bool on = t < nv && p0 + p < a.P;
                s.v[t][p] = on ? ldf(vp + t * a.v.token + p) : 0.0f;
                s.dy[t][p] = on ? ldf(yp + t * a.dy.token + p) : 0.0f;
            }
            const int64_t at = ((b * a.H + h) * w.chunks + chunk) * a.N * a.P + p0;
#pragma unroll
            for (int u = 0; u < NP * kPT / 256; u++) {
                const int e = tid + 256 * u, n = e / kPT, p = e % kPT;
                const bool on = n < a.N && p0 + p < a.P;
                const float hv = on ? w.before[at + n * a.P + p] : 0.0f, rv = on ? w.after[at + n * a.P + p] : 0.0f;
                s.H[n][p] = hv;
                s.R[n][p] = rv;
                through = fmaf(hv, rv, through);
            }
            __syncthreads();
            {  // scores
                float qk[4][4], yv[4][4];
                auto scores = [&](float (&out)[4][4], const auto& left, const auto& right, int n) {  // rows . rows, of n values
                    float2 acc[4][4] = {};
                    for (int e = 0; e < n; e += 4) {
                        float4 x[4], z[4];
#pragma unroll
                        for (int r = 0; r < 4; r++) x[r] = at4(&left[ty + 16 * r][e]), z[r] = at4(&right[tx + 16 * r][e]);
#pragma unroll
                        for (int r = 0; r < 4; r++)
#pragma unroll
                            for (int c = 0; c < 4; c++) dot4(acc[r][c], x[r], z[c]);
                    }
#pragma unroll
                    for (int r = 0; r < 4; r++)
#pragma unroll
                        for (int c = 0; c < 4; c++) out[r][c] = acc[r][c].x + acc[r][c].y;
                };
                scores(qk, s.q, s.k, NP);
                scores(yv, s.dy, s.v, kPT);
                float col[4] = {};
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int i = ty + 16 * r;
                    float row = 0.0f;
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        const int j = tx + 16 * c;
                        const float m = j <= i ? a.scale * ex2(two_diff(s.c[i], s.c[j])) : 0.0f;
                        const float e = yv[r][c] * m;
                        s.E[i][j] = e;
                        s.S[i][j] = qk[r][c] * m;
                        const float wv = j < i ? e * qk[r][c] : 0.0f;
                        row += wv;
                        col[c] += wv;
                    }
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) row += __shfl_xor_sync(kFull, row, o);
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
            {  // dv, and b from its inter-chunk part: rows 4 ty + r, columns 4 tx + c
                float2 in[4][2] = {}, ac[4][2] = {};
#pragma unroll 4
                for (int i = 0; i < nc; i++) {
                    const float4 x = at4(&s.S[i][4 * ty]), z = at4(&s.dy[i][4 * tx]);
                    const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int r = 0; r < 4; r++) fma4(ac[r], xs[r], z);
                }
                for (int n = 0; n < NP; n += 4) {
                    float4 x[4], z[4];
#pragma unroll
                    for (int r = 0; r < 4; r++) x[r] = at4(&s.k[4 * ty + r][n]), z[r] = at4(&s.R[n + r][4 * tx]);
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        fma4(in[r], x[r].x, z[0]);
                        fma4(in[r], x[r].y, z[1]);
                        fma4(in[r], x[r].z, z[2]);
                        fma4(in[r], x[r].w, z[3]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int j = 4 * ty + r;
                    const float d = ex2(two_diff(cl, s.c[j]));
                    float bj = 0.0f;
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        const int p = 4 * tx + c;
                        const float x = d * (c & 1 ? in[r][c / 2].y : in[r][c / 2].x);
                        bj = fmaf(s.v[j][p], x, bj);
                        if (j < nt && p0 + p < a.P)
                            st(static_cast<T*>(w.dv) + ((b * a.L + t0 + j) * a.H + h) * a.P + p0 + p,
                               j < nv ? (c & 1 ? ac[r][c / 2].y : ac[r][c / 2].x) + x : 0.0f);
                    }
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) bj += __shfl_xor_sync(kFull, bj, o);
                    if (tx == 0) s.b[j] += bj;
                }
            }
            {  // dq, and a from its inter-chunk part: rows 4 ty + r, columns tx + 16 n
                float2 ac[4][NB] = {}, in[4][NB] = {};
                for (int j = 0; j < nc; j += 4) {
                    float4 x[4];
#pragma unroll
                    for (int r = 0; r < 4; r++) x[r] = at4(&s.E[4 * ty + r][j]);
#pragma unroll
                    for (int n = 0; n < NB; n++) {
                        const int m = tx + 16 * n;
                        const float4 z = make_float4(s.k[j][m], s.k[j + 1][m], s.k[j + 2][m], s.k[j + 3][m]);
#pragma unroll
                        for (int r = 0; r < 4; r++) dot4(ac[r][n], x[r], z);
                    }
                }
                for (int p = 0; p < kPT; p += 4) {
                    float4 x[4];
#pragma unroll
                    for (int r = 0; r < 4; r++) x[r] = at4(&s.dy[4 * ty + r][p]);
#pragma unroll
                    for (int n = 0; n < NB; n++) {
                        const float4 z = at4(&s.H[tx + 16 * n][p]);
#pragma unroll
                        for (int r = 0; r < 4; r++) dot4(in[r][n], x[r], z);
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int i = 4 * ty + r;
                    const float d = a.scale * ex2(s.c[i].h + s.c[i].l);
                    float ai = 0.0f;
#pragma unroll
                    for (int n = 0; n < NB; n++) {
                        const float x = d * (in[r][n].x + in[r][n].y);
                        ai = fmaf(s.q[i][tx + 16 * n], x, ai);
                        dq[r][n] += ac[r][n].x + ac[r][n].y + x;
                    }
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) ai += __shfl_xor_sync(kFull, ai, o);
                    if (tx == 0) s.a[i] += ai;
                }
            }
            {  // dk, like dq
#pragma unroll 4
                for (int i = 0; i < nc; i++) {
                    const float4 x = at4(&s.E[i][4 * ty]);
#pragma unroll
                    for (int n = 0; n < NB; n++) {
                        const float z = s.q[i][tx + 16 * n];
                        dk[0][n] = fma2(make_float2(x.x, x.y), splat2(z), dk[0][n]);
                        dk[1][n] = fma2(make_float2(x.z, x.w), splat2(z), dk[1][n]);
                    }
                }
                float2 in[4][NB] = {};
                for (int p = 0; p < kPT; p += 4) {
                    float4 x[4];
#pragma unroll
                    for (int r = 0; r < 4; r++) x[r] = at4(&s.v[4 * ty + r][p]);
#pragma unroll
                    for (int n = 0; n < NB; n++) {
                        const float4 z = at4(&s.R[tx + 16 * n][p]);
#pragma unroll
                        for (int r = 0; r < 4; r++) dot4(in[r][n], x[r], z);
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    const float2 d = make_float2(ex2(two_diff(cl, s.c[4 * ty + r])), ex2(two_diff(cl, s.c[4 * ty + r + 1])));
#pragma unroll
                    for (int n = 0; n < NB; n++)
                        dk[r / 2][n] = fma2(d, make_float2(in[r][n].x + in[r][n].y, in[r + 1][n].x + in[r + 1][n].y), dk[r / 2][n]);
                }
            }
        }
        // dg of this head
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) through += __shfl_xor_sync(kFull, through, o);
        if (lane == 0) s.red[warp] = through;
        __syncthreads();
        if (warp == 0) {
            float sum = 0.0f;
#pragma unroll
            for (int u = 0; u < 8; u++) sum += s.red[u];
            const Two cl = s.c[C - 1];
            sum *= ex2(cl.h + cl.l);
            const float a0 = s.a[2 * lane], a1 = s.a[2 * lane + 1], b0 = s.b[2 * lane], b1 = s.b[2 * lane + 1];
            float A = a0 + a1, B = b0 + b1;  // suffix of a, prefix of b over lanes
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float x = __shfl_down_sync(kFull, A, o), y = __shfl_up_sync(kFull, B, o);
                if (lane + o < 32) A += x;
                if (lane >= o) B += y;
            }
            const float Bx = __shfl_up_sync(kFull, B, 1), Ax = __shfl_down_sync(kFull, A, 1);
            const float pre = lane > 0 ? Bx : 0.0f, suf = lane < 31 ? Ax : 0.0f;
            const float g0 = (a0 + a1 + suf) + pre + sum, g1 = (a1 + suf) + (pre + b0) + sum;
            const int t = 2 * lane;
            if (t < nt) w.dg[(b * a.L + t0 + t) * a.H + h] = t < nv ? g0 : 0.0f;
            if (t + 1 < nt) w.dg[(b * a.L + t0 + t + 1) * a.H + h] = t + 1 < nv ? g1 : 0.0f;
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
            const int64_t at = ((b * a.L + t0 + t) * a.G + gq) * a.N + c;
            const float x = t < nv ? dq[r][n] : 0.0f, z = t < nv ? (r & 1 ? dk[r / 2][n].y : dk[r / 2][n].x) : 0.0f;
            if (w.splits > 1) {
                const int64_t part = split * a.Bsz * a.L * a.G * a.N + at;
                w.dq_part[part] = x;
                w.dk_part[part] = z;
            } else {
                st(static_cast<T*>(w.dq) + at, x);
                st(static_cast<T*>(w.dk) + at, z);
            }
        }
    }
}

// Four values a thread (n is a multiple of 4, VEC) or one; parts in a fixed order.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_sum_parts(const float* part, T* out, const float* part2, T* out2, int splits, int64_t n) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * (VEC ? 4 : 1);
    if (i >= n) return;
    if (blockIdx.y) {
        part = part2;
        out = out2;
    }
    if (VEC) {
        float4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int k = 0; k < splits; k++) {
            const float4 x = *reinterpret_cast<const float4*>(part + k * n + i);
            s = {s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w};
        }
        st(out + i, s.x);
        st(out + i + 1, s.y);
        st(out + i + 2, s.z);
        st(out + i + 3, s.w);
    } else {
        float s = 0.0f;
        for (int k = 0; k < splits; k++) s += part[k * n + i];
        st(out + i, s);
    }
}

// part[slice, h] = sum of the slice's rows (32 heads x 8 rows at a time)
__global__ void __launch_bounds__(256) k_sum_rows(const float* x, float* part, int64_t rows, int64_t H) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t h = (int64_t)blockIdx.x * 32 + lane;
    const int64_t per = (rows + gridDim.y - 1) / gridDim.y;
    const int64_t lo = blockIdx.y * per, hi = min(rows, lo + per);
    float v = 0.0f;
    if (h < H)
        for (int64_t r = lo + warp; r < hi; r += 8) v += x[r * H + h];
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && h < H) {
        float t = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; u++) t += s[u][lane];
        part[blockIdx.y * H + h] = t;
    }
}

template <typename T, int NR> cudaError_t walk_mode(const WalkArgs& w, bool sum, cudaStream_t st) {
    const Args& a = w.a;
    const int64_t segs = sum && w.dirs == 1 ? w.plan.K - 1 : w.plan.K;
    const unsigned grid = (unsigned)(ceil_div(a.P, kWalkP) * a.H * a.Bsz * w.dirs * segs);
    if (sum) k_sum32<T, NR / 2><<<grid, 256, 0, st>>>(w);
    else k_walk32<T, NR><<<grid, 256, 0, st>>>(w);
    return cudaGetLastError();
}

template <typename T> cudaError_t walk_io(const WalkArgs& w, bool sum, cudaStream_t st) {
    if (w.a.N <= 32) return walk_mode<T, 4>(w, sum, st);
    if (w.a.N <= 64) return walk_mode<T, 8>(w, sum, st);
    return walk_mode<T, 16>(w, sum, st);
}

template <typename T, int NB> cudaError_t bwd_n(const BwdArgs& b, cudaStream_t st) {
    const int bytes = (int)sizeof(Smem32<NB>);
    const cudaError_t e = allow_smem<k_bwd32<T, NB>>(bytes);
    if (e != cudaSuccess) return e;
    k_bwd32<T, NB><<<(unsigned)(b.a.Bsz * b.chunks * b.a.G * b.splits), 256, bytes, st>>>(b);
    return cudaGetLastError();
}

template <typename T> cudaError_t bwd_io(const BwdArgs& b, cudaStream_t st) {
    if (b.a.N <= 32) return bwd_n<T, 2>(b, st);
    if (b.a.N <= 64) return bwd_n<T, 4>(b, st);
    return bwd_n<T, 8>(b, st);
}

}  // namespace

// Whether every run of four values of q, k, v, dy and the states is whole and aligned.
static bool fours(const WalkArgs& w) {
    const Args& a = w.a;
    const uintptr_t bytes = a.dtype == 0 ? 16 : 8;
    for (const In* x : {&a.q, &a.k, &a.v, &a.dy})
        if (reinterpret_cast<uintptr_t>(x->p) % bytes != 0 || x->token % 4 != 0 || x->batch % 4 != 0) return false;
    return a.N % 4 == 0 && a.P % 4 == 0;
}

cudaError_t launch_walk32(const WalkArgs& args, bool sum, cudaStream_t st) {
    WalkArgs w = args;
    w.vec = fours(w);
    if (w.a.dtype == 0) return walk_io<float>(w, sum, st);
    if (w.a.dtype == 1) return walk_io<__half>(w, sum, st);
    return walk_io<__nv_bfloat16>(w, sum, st);
}

cudaError_t launch_carry32(const WalkArgs& w, cudaStream_t st) {
    // grid.y: at most 2^16 - 1 (direction, batch row, head) units a launch
    const int64_t units = w.dirs * w.a.Bsz * w.a.H;
    for (int64_t at = 0; at < units; at += 65535) {
        const int64_t n = units - at < 65535 ? units - at : 65535;
        k_carry32<<<dim3((unsigned)ceil_div(w.a.N * w.a.P, 256), (unsigned)n), 256, 0, st>>>(w, at);
    }
    return cudaGetLastError();
}

cudaError_t launch_bwd32(const BwdArgs& b, cudaStream_t st) {
    if (b.a.dtype == 0) return bwd_io<float>(b, st);
    if (b.a.dtype == 1) return bwd_io<__half>(b, st);
    return bwd_io<__nv_bfloat16>(b, st);
}

template <typename T>
cudaError_t sum_parts(const float* part, void* out, const float* part2, void* out2, int splits, int64_t n, cudaStream_t st) {
    const bool vec = n % 4 == 0;
    const dim3 grid((unsigned)ceil_div(n, vec ? 1024 : 256), out2 ? 2 : 1);
    T *o = static_cast<T*>(out), *o2 = static_cast<T*>(out2);
    if (vec) k_sum_parts<T, true><<<grid, 256, 0, st>>>(part, o, part2, o2, splits, n);
    else k_sum_parts<T, false><<<grid, 256, 0, st>>>(part, o, part2, o2, splits, n);
    return cudaGetLastError();
}
cudaError_t launch_sum_parts(const float* part, void* out, const float* part2, void* out2, int splits, int64_t n, int dtype,
                             cudaStream_t st) {
    if (dtype == 0) return sum_parts<float>(part, out, part2, out2, splits, n, st);
    if (dtype == 1) return sum_parts<__half>(part, out, part2, out2, splits, n, st);
    return sum_parts<__nv_bfloat16>(part, out, part2, out2, splits, n, st);
}

cudaError_t launch_sum_rows(const float* dg, float* part, float* out, int64_t rows, int64_t H, cudaStream_t st) {
    const unsigned gx = (unsigned)ceil_div(H, 32);
    k_sum_rows<<<dim3(gx, kDgParts), 256, 0, st>>>(dg, part, rows, H);
    k_sum_rows<<<dim3(gx, 1), 256, 0, st>>>(part, out, kDgParts, H);
    return cudaGetLastError();
}

}  // namespace la
}  // namespace ss
