// Group norm of each token's channels with an activation, forward and backward.
//
// Both directions are bound by HBM: x, z (and dout) are read once into
// registers, the statistics are two sums over the registers (mean, then the
// squared deviations: no cancellation), and the results are written once.  A
// thread keeps its channels' weight and bias (and, in the backward, their
// gradients' sums) while it walks over rows, so parameters are not re-read and
// the parameter gradients need one small second pass.
#include "la_dev.cuh"
#include "ss_la.h"

namespace ss {
namespace {

using la::ex2;
using la::kLog2e;

template <typename T, int E> struct Vec;  // E values moved at once
template <> struct Vec<float, 4> { using M = uint4; };
template <> struct Vec<__half, 8> { using M = uint4; };
template <> struct Vec<__nv_bfloat16, 8> { using M = uint4; };
template <typename T> struct Vec<T, 1> { using M = T; };

template <typename T, int E> __device__ __forceinline__ typename Vec<T, E>::M load(const void* p, int64_t i) {
    return *reinterpret_cast<const typename Vec<T, E>::M*>(static_cast<const T*>(p) + i);
}
template <typename T, int E> __device__ __forceinline__ void widen(const typename Vec<T, E>::M& m, float (&f)[E]) {
    union {
        typename Vec<T, E>::M m;
        T t[E];
    } u;
    u.m = m;
#pragma unroll
    for (int e = 0; e < E; e++) f[e] = la::ldf(&u.t[e]);
}
template <typename T, int E> __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[E]) {
    union {
        typename Vec<T, E>::M m;
        T t[E];
    } u;
#pragma unroll
    for (int e = 0; e < E; e++) st(&u.t[e], f[e]);
    *reinterpret_cast<typename Vec<T, E>::M*>(static_cast<T*>(p) + i) = u.m;
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + ex2(-kLog2e * x)); }

// Sum over the LPG threads of a group (all of them get it): lanes of a warp, or the block.
template <int LPG> __device__ __forceinline__ float group_sum(float v, float* red) {
    constexpr int W = LPG < 32 ? LPG : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if (LPG > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < LPG / 32; w++) v += red[w];
    }
    return v;
}

// LPG threads hold one group, VPT runs of E values each.  LPG <= 32: a warp
// covers 32 / LPG adjacent groups, a block's 8 warps take different rows.
// LPG > 32: the block covers one group.  Rows advance by gridDim.y * (rows per step).
template <int LPG> constexpr int kThreads = LPG <= 32 ? 256 : LPG;
template <int LPG> constexpr int kRowsPerStep = LPG <= 32 ? 8 : 1;

template <typename T, int E, int LPG, int VPT, bool BWD>
__global__ void __launch_bounds__(kThreads<LPG>) k_gnorm(GnormArgs a) {
    __shared__ float red[32];
    __shared__ float cols[BWD && LPG <= 32 ? 8 : 1][BWD && LPG <= 32 ? 32 * E * VPT : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t gs = a.C / a.groups;
    const int nvec = (int)(gs / E);
    const int64_t slot = LPG <= 32 ? (int64_t)blockIdx.x * 32 + lane : (int64_t)blockIdx.x * LPG + threadIdx.x;
    const int64_t grp = slot / LPG;
    const int l = (int)(slot % LPG);
    const bool center = a.flags & SS_GNORM_CENTER, first = a.flags & SS_GNORM_GATE_FIRST;
    const bool gate = a.z != nullptr;
    const float inv = 1.0f / (float)gs;
    bool on[VPT];
    float w[VPT][E], bb[VPT][E], dw[VPT][E], db[VPT][E];
#pragma unroll
    for (int j = 0; j < VPT; j++) {
        on[j] = grp < a.groups && l + j * LPG < nvec;
        const int64_t c = grp * gs + (int64_t)(l + j * LPG) * E;
#pragma unroll
        for (int e = 0; e < E; e++) {
            w[j][e] = on[j] && a.weight ? a.weight[c + e] : 1.0f;
            bb[j][e] = on[j] && a.bias ? a.bias[c + e] : 0.0f;
            dw[j][e] = db[j][e] = 0.0f;
        }
    }
    // the runs of one row, on their way while the row before is computed (one run
    // a thread; threads with several have enough loads in flight)
    using M = typename Vec<T, E>::M;
    constexpr bool kAhead = VPT == 1;
    M xn[VPT], zn[VPT], dn[VPT];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int j = 0; j < VPT; j++)
            if (r < a.M && on[j]) {
                const int64_t i = r * a.C + grp * gs + (int64_t)(l + j * LPG) * E;
                xn[j] = load<T, E>(a.x, i);
                if (gate) zn[j] = load<T, E>(a.z, i);
                if (BWD) dn[j] = load<T, E>(a.dout, i);
            }
    };
    const int64_t pace = (int64_t)gridDim.y * kRowsPerStep<LPG>, mine = LPG <= 32 ? warp : 0;
    int64_t r0 = (int64_t)blockIdx.y * kRowsPerStep<LPG>;
    if (kAhead) fetch(r0 + mine);
    for (; r0 < a.M; r0 += pace) {
        const int64_t r = r0 + mine;
        const bool row = r < a.M;
        const int64_t at = r * a.C + grp * gs;
        float x[VPT][E], z[VPT][E], d[VPT][E];
        if (!kAhead) fetch(r);
#pragma unroll
        for (int j = 0; j < VPT; j++) {
            if (row && on[j]) {
                widen<T, E>(xn[j], x[j]);
                if (gate) widen<T, E>(zn[j], z[j]);
                if (BWD) widen<T, E>(dn[j], d[j]);
            } else {
#pragma unroll
                for (int e = 0; e < E; e++) x[j][e] = z[j][e] = d[j][e] = 0.0f;
            }
        }
        if (kAhead) fetch(r + pace);
        // u: what is normalised (x, or x silu(z))
        float u[VPT][E], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; j++)
#pragma unroll
            for (int e = 0; e < E; e++) {
                u[j][e] = gate && first ? x[j][e] * (z[j][e] * sigmoid(z[j][e])) : x[j][e];
                sum += u[j][e];
            }
        const float mean = center ? group_sum<LPG>(sum, red) * inv : 0.0f;
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; j++)
#pragma unroll
            for (int e = 0; e < E; e++) {
                u[j][e] -= mean;
                sq += on[j] ? u[j][e] * u[j][e] : 0.0f;
            }
        const float rstd = rsqrtf(group_sum<LPG>(sq, red) * inv + a.eps);
        if (!BWD) {
#pragma unroll
            for (int j = 0; j < VPT; j++) {
                float o[E];
#pragma unroll
                for (int e = 0; e < E; e++) {
                    const float n = fmaf(u[j][e] * rstd, w[j][e], bb[j][e]);
                    o[e] = gate ? (first ? n : n * (z[j][e] * sigmoid(z[j][e]))) : n * sigmoid(n);
                }
                if (row && on[j]) store<T, E>(a.out, at + (int64_t)(l + j * LPG) * E, o);
            }
        } else {
            float s1 = 0.0f, s2 = 0.0f;  // sums of t and t * xhat, t the gradient of xhat
#pragma unroll
            for (int j = 0; j < VPT; j++) {
                float o[E];
#pragma unroll
                for (int e = 0; e < E; e++) {
                    const float xh = u[j][e] * rstd;
                    const float n = fmaf(xh, w[j][e], bb[j][e]);
                    float g = d[j][e];
                    if (gate && !first) {
                        const float sg = sigmoid(z[j][e]);
                        o[e] = g * n * (sg * (1.0f + z[j][e] * (1.0f - sg)));
                        g *= z[j][e] * sg;
                    } else if (!gate) {
                        const float sg = sigmoid(n);
                        g *= sg * (1.0f + n * (1.0f - sg));
                    }
                    dw[j][e] = fmaf(g, xh, dw[j][e]);
                    db[j][e] += g;
                    const float t = g * w[j][e];
                    s1 += t;
                    s2 = fmaf(t, xh, s2);
                    d[j][e] = t;
                    u[j][e] = xh;
                }
                if (gate && !first && row && on[j]) store<T, E>(a.dz, at + (int64_t)(l + j * LPG) * E, o);
            }
            s1 = center ? group_sum<LPG>(s1, red) * inv : 0.0f;
            s2 = group_sum<LPG>(s2, red) * inv;
#pragma unroll
            for (int j = 0; j < VPT; j++) {
                float o[E], o2[E];
#pragma unroll
                for (int e = 0; e < E; e++) {
                    const float du = rstd * (d[j][e] - s1 - u[j][e] * s2);
                    o[e] = du;
                    if (gate && first) {
                        const float sg = sigmoid(z[j][e]);
                        o2[e] = du * x[j][e] * (sg * (1.0f + z[j][e] * (1.0f - sg)));
                        o[e] = du * (z[j][e] * sg);
                    }
                }
                const int64_t i = at + (int64_t)(l + j * LPG) * E;
                if (row && on[j]) {
                    store<T, E>(a.dx, i, o);
                    if (gate && first) store<T, E>(a.dz, i, o2);
                }
            }
        }
    }
    if (BWD) {
        // this block's rows' sums of dweight and dbias: part[blockIdx.y][0 and 1][C]
        float* part = a.part + (int64_t)blockIdx.y * 2 * a.C;
#pragma unroll
        for (int pass = 0; pass < 2; pass++) {
            if (LPG <= 32) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < VPT; j++)
#pragma unroll
                    for (int e = 0; e < E; e++) cols[warp][(j * E + e) * 32 + lane] = pass ? db[j][e] : dw[j][e];
                __syncthreads();
                if (warp != 0) continue;
            }
#pragma unroll
            for (int j = 0; j < VPT; j++)
                if (on[j]) {
                    const int64_t c = grp * gs + (int64_t)(l + j * LPG) * E;
#pragma unroll
                    for (int e = 0; e < E; e++) {
                        float v = pass ? db[j][e] : dw[j][e];
                        if (LPG <= 32) {
                            v = 0.0f;
#pragma unroll
                            for (int k = 0; k < 8; k++) v += cols[k][(j * E + e) * 32 + lane];
                        }
                        part[pass * a.C + c + e] = v;
                    }
                }
        }
    }
}

// dweight, dbias: sums of the blocks' parts, 32 channels x 8 runs of blocks per block
__global__ void __launch_bounds__(256) k_gnorm_params(const float* part, float* dweight, float* dbias, int64_t C, int64_t blocks) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < 2 * C)
        for (int64_t k = warp; k < blocks; k += 8) v += part[k * 2 * C + c];
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < 2 * C) {
        float t = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; u++) t += s[u][lane];
        float* out = c < C ? dweight : dbias;
        if (out) out[c < C ? c : c - C] = t;
    }
}

// Row blocks of a launch: enough blocks for a few on every SM.
int64_t row_blocks(int64_t M, int64_t xblocks, int64_t rows, int64_t per_sm) {
    const int64_t want = ceil_div(la::kSms * per_sm, xblocks), most = ceil_div(M, rows);
    const int64_t y = want < most ? want : most;
    return y < 1 ? 1 : (y > 65535 ? 65535 : y);
}

template <typename T, int E, int LPG, int VPT, bool BWD> cudaError_t go(const GnormArgs& a, cudaStream_t st) {
    const int64_t x = LPG <= 32 ? ceil_div(a.groups * LPG, 32) : a.groups;
    const int64_t y = BWD ? gnorm_bwd_blocks(a.M, a.C, a.groups)
                          : row_blocks(a.M, x, kRowsPerStep<LPG>, LPG <= 32 ? 16 : 8);
    k_gnorm<T, E, LPG, VPT, BWD><<<dim3((unsigned)x, (unsigned)y), kThreads<LPG>, 0, st>>>(a);
    return cudaGetLastError();
}

bool aligned(const GnormArgs& a) {
    const void* p[] = {a.x, a.z, a.dout, a.out, a.dx, a.dz};
    for (const void* q : p)
        if (reinterpret_cast<uintptr_t>(q) & 15u) return false;
    return true;
}

// The threads that hold a group, by the number of 16-byte runs in it; groups
// that are no whole number of runs move value by value.
template <typename T, bool BWD> cudaError_t pick(const GnormArgs& a, cudaStream_t st) {
    constexpr int E = 16 / (int)sizeof(T);
    const int64_t gs = a.C / a.groups;
    if (gs % E != 0 || !aligned(a)) {
        if (gs <= 256) return go<T, 1, 32, 8, BWD>(a, st);
        if (gs <= 2048) return go<T, 1, 256, 8, BWD>(a, st);
        return go<T, 1, 512, 16, BWD>(a, st);
    }
    const int64_t n = gs / E;
    if (n <= 4) return go<T, E, 4, 1, BWD>(a, st);
    if (n <= 8) return go<T, E, 8, 1, BWD>(a, st);
    if (n <= 16) return go<T, E, 16, 1, BWD>(a, st);
    if (n <= 32) return go<T, E, 32, 1, BWD>(a, st);
    if (n <= 64) return go<T, E, 32, 2, BWD>(a, st);
    if (n <= 256) return go<T, E, 256, 1, BWD>(a, st);
    if (n <= 512) return go<T, E, 256, 2, BWD>(a, st);
    if (n <= 1024) return go<T, E, 256, 4, BWD>(a, st);
    return go<T, E, 512, 4, BWD>(a, st);
}

template <bool BWD> cudaError_t pick_io(const GnormArgs& a, cudaStream_t st) {
    if (a.dtype == 0) return pick<float, BWD>(a, st);
    if (a.dtype == 1) return pick<__half, BWD>(a, st);
    return pick<__nv_bfloat16, BWD>(a, st);
}

}  // namespace

// Row blocks of the backward, a function of the sizes alone (the workspace
// holds one partial sum per block): by the channels a block covers at most.
int64_t gnorm_bwd_blocks(int64_t M, int64_t C, int64_t groups) {
    const int64_t gs = C / groups;
    const int64_t x = gs > 256 ? groups : ceil_div(C, 256);
    return row_blocks(M, x, gs > 256 ? 1 : 8, 8);
}

cudaError_t launch_gnorm_fwd(const GnormArgs& a, cudaStream_t st) { return pick_io<false>(a, st); }

cudaError_t launch_gnorm_bwd(const GnormArgs& a, cudaStream_t st) {
    const cudaError_t e = pick_io<true>(a, st);
    if (e != cudaSuccess) return e;
    k_gnorm_params<<<(unsigned)ceil_div(2 * a.C, 32), 256, 0, st>>>(a.part, a.dweight, a.dbias, a.C,
                                                                   gnorm_bwd_blocks(a.M, a.C, a.groups));
    return cudaGetLastError();
}

}  // namespace ss
