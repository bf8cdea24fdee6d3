// Group norm of each token's channels with an activation, forward and backward.
//
// Both directions are bound by HBM: x, z (and dout) are read once into
// registers, the statistics are two sums over the registers (mean, then the
// squared deviations: no cancellation), and the results are written once.  A
// thread keeps its channels while it walks over rows, so that weight and bias stay
// in registers (or the L1 cache), and the parameter gradients need one small second
// pass.  Sums and statistics are f32.
//
// Measured, bf16 with a gate (503 MB forward, 419 MB backward; copying takes 74 and
// 62 us): 16384 x 5120 in groups of 64: 82 us, backward of 8192 rows 81 us; groups of
// 512: 101 and 116, of 1024: 109 and 144, of 5120: 127 and 138 (one row in work a
// block or warp, and a barrier a sum: nothing covers a row's reductions).
#include "../simd.cuh"
#include "la_dev.cuh"
#include "ss_la.h"

namespace ss {
namespace {

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

__device__ __forceinline__ float sigmoid(float x) { return rcpa(1.0f + ex2a(-kLog2e * x)); }
__device__ __forceinline__ float2 sigmoid(float2 x) {
    const float2 e = mul2(x, splat2(-kLog2e));
    const float2 d = add2(make_float2(ex2a(e.x), ex2a(e.y)), splat2(1.0f));
    return make_float2(rcpa(d.x), rcpa(d.y));
}
// A run's values as pairs (runs of one value: the second of the pair is not used)
template <int E> __device__ __forceinline__ float2 pair(const float (&x)[E], int e) {
    return make_float2(x[e], E > 1 ? x[e + (E > 1)] : 0.0f);
}
template <int E> __device__ __forceinline__ void put(float (&x)[E], int e, float2 v) {
    x[e] = v.x;
    if (E > 1) x[e + (E > 1)] = v.y;
}

// Sum over the threads of a group (all of them get it): LPG lanes of a warp, or
// the whole block (LPG = 0) by way of red, 32 floats that no other sum since the
// last barrier but one has used.
template <int LPG> __device__ __forceinline__ float group_sum(float v, float* red) {
    constexpr int W = LPG > 0 ? LPG : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if (LPG == 0) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < (int)blockDim.x / 32 ? red[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    }
    return v;
}
// Two sums at once.
template <int LPG> __device__ __forceinline__ float2 group_sum2(float2 v, float* red, float* red2) {
    constexpr int W = LPG > 0 ? LPG : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v = add2(v, make_float2(__shfl_xor_sync(kFull, v.x, o), __shfl_xor_sync(kFull, v.y, o)));
    if (LPG == 0) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) {
            red[threadIdx.x >> 5] = v.x;
            red2[threadIdx.x >> 5] = v.y;
        }
        __syncthreads();
        const bool on = lane < (int)blockDim.x / 32;
        v = make_float2(on ? red[lane] : 0.0f, on ? red2[lane] : 0.0f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = add2(v, make_float2(__shfl_xor_sync(kFull, v.x, o), __shfl_xor_sync(kFull, v.y, o)));
    }
    return v;
}

// A group is held by LPG lanes of a warp, VPT runs of E values each: a warp
// covers 32 / LPG adjacent groups, the 8 warps of a block take different rows.
// LPG = 0: the block covers one group of one row.  Rows advance by gridDim.y *
// kRowsPerStep.
template <int LPG> constexpr int kRowsPerStep = LPG > 0 ? 8 : 1;

// Threads whose runs are of 16 bytes keep the rows to come on their way to shared
// memory (their own slots of it: no barrier), as many as it takes to cover the
// memory's latency.
template <int E> constexpr bool kRing = E > 1;
template <int LPG, int VPT, bool BWD> constexpr int kDepth = LPG == 0 && VPT > 2 ? 2 : (VPT > 1 || BWD ? 3 : 4);
// Blocks that are to fit on an SM: by their registers.
template <int LPG, int VPT, bool BWD>
constexpr int kPerSm = LPG > 0 ? (VPT == 1 ? (BWD ? 2 : 4) : (BWD || VPT > 4 ? 1 : 2)) : (VPT > 1 || BWD ? 1 : 2);
__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T, int E, int LPG, int VPT, bool BWD>
__global__ void __launch_bounds__(LPG > 0 ? 256 : (VPT <= 2 ? 640 : 512), kPerSm<LPG, VPT, BWD>) k_gnorm(GnormArgs a) {
    extern __shared__ __align__(16) uint4 ring[];  // [depth][x, z, dout][run][thread] (kRing)
    __shared__ float s_red[LPG > 0 ? 1 : 2][4][32];  // of rows by turns
    __shared__ float cols[BWD && LPG > 0 ? 8 : 1][BWD && LPG > 0 ? 32 * E * VPT : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t gs = a.C / a.groups;
    const int nvec = (int)(gs / E);
    const int64_t slot = (int64_t)blockIdx.x * 32 + lane;
    const int lanes = LPG > 0 ? LPG : (int)blockDim.x;
    const int64_t grp = LPG > 0 ? slot / lanes : (int64_t)blockIdx.x;
    const int l = LPG > 0 ? (int)(slot % lanes) : (int)threadIdx.x;
    const bool center = a.flags & SS_GNORM_CENTER, first = a.flags & SS_GNORM_GATE_FIRST;
    const bool gate = a.z != nullptr;
    const float inv = 1.0f / (float)gs;
    bool on[VPT];
    // weight and bias: in registers with one run a thread, read again for each row (from the L1 cache) with several
    float w[1][E], bb[1][E], dw[VPT][E], db[VPT][E];
    auto params = [&](int j, float (&wj)[E], float (&bj)[E]) {
        const int64_t c = grp * gs + (int64_t)(l + j * lanes) * E;
        auto get = [&](const float* p, float other, float (&f)[E]) {
            if (!p || !on[j]) {
#pragma unroll
                for (int e = 0; e < E; e++) f[e] = other;
            } else if constexpr (E == 1) {
                f[0] = __ldg(p + c);
            } else {
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const float4 x = __ldg(reinterpret_cast<const float4*>(p + c + e));
                    f[e] = x.x;
                    f[e + 1] = x.y;
                    f[e + 2] = x.z;
                    f[e + 3] = x.w;
                }
            }
        };
        get(a.weight, 1.0f, wj);
        get(a.bias, 0.0f, bj);
    };
#pragma unroll
    for (int j = 0; j < VPT; j++) {
        on[j] = grp < a.groups && l + j * lanes < nvec;
#pragma unroll
        for (int e = 0; e < E; e++) dw[j][e] = db[j][e] = 0.0f;
    }
    if (VPT == 1) params(0, w[0], bb[0]);
    const int64_t pace = (int64_t)gridDim.y * kRowsPerStep<LPG>, mine = LPG > 0 ? warp : 0;
    int64_t r0 = (int64_t)blockIdx.y * kRowsPerStep<LPG>;
    constexpr int D = kDepth<LPG, VPT, BWD>, kIn = BWD ? 3 : 2;
    auto at_ring = [&](int stage, int which, int j) {
        return ring + ((stage * kIn + which) * VPT + j) * (int)blockDim.x + threadIdx.x;
    };
    auto ahead = [&](int stage, int64_t r) {
#pragma unroll
        for (int j = 0; j < VPT; j++)
            if (r < a.M && on[j]) {
                const int64_t i = r * a.C + grp * gs + (int64_t)(l + j * lanes) * E;
                copy16(at_ring(stage, 0, j), static_cast<const T*>(a.x) + i);
                if (gate) copy16(at_ring(stage, 1, j), static_cast<const T*>(a.z) + i);
                if (BWD) copy16(at_ring(stage, 2, j), static_cast<const T*>(a.dout) + i);
            }
        copy_commit();
    };
    if constexpr (kRing<E>) {
#pragma unroll
        for (int i = 0; i < D - 1; i++) ahead(i, r0 + i * pace + mine);
    }
    int stage = 0, turn = 0;
    for (; r0 < a.M; r0 += pace) {
        float(*red)[32] = s_red[turn];
        if (LPG == 0) turn ^= 1;
        const int64_t r = r0 + mine;
        const bool row = r < a.M;
        const int64_t at = r * a.C + grp * gs;
        float x[VPT][E], z[VPT][E], d[VPT][E];
        if constexpr (kRing<E>) {
            ahead(stage == 0 ? D - 1 : stage - 1, r + (D - 1) * pace);
            copy_wait<D - 1>();
        }
#pragma unroll
        for (int j = 0; j < VPT; j++) {
            const int64_t i = at + (int64_t)(l + j * lanes) * E;
            if (row && on[j]) {
                if constexpr (kRing<E>) {
                    widen<T, E>(*at_ring(stage, 0, j), x[j]);
                    if (gate) widen<T, E>(*at_ring(stage, 1, j), z[j]);
                    if (BWD) widen<T, E>(*at_ring(stage, 2, j), d[j]);
                } else {
                    widen<T, E>(load<T, E>(a.x, i), x[j]);
                    if (gate) widen<T, E>(load<T, E>(a.z, i), z[j]);
                    if (BWD) widen<T, E>(load<T, E>(a.dout, i), d[j]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; e++) x[j][e] = z[j][e] = d[j][e] = 0.0f;
            }
        }
        if constexpr (kRing<E>) stage = stage + 1 == D ? 0 : stage + 1;
        // u: what is normalised (x, or x silu(z))
        float u[VPT][E];
        float2 sum = splat2(0.0f);
#pragma unroll
        for (int j = 0; j < VPT; j++)
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                float2 v = pair(x[j], e);
                if (gate && first) {
                    const float2 zv = pair(z[j], e);
                    v = mul2(v, mul2(zv, sigmoid(zv)));
                }
                sum = add2(sum, v);
                put(u[j], e, v);
            }
        const float mean = center ? group_sum<LPG>(sum.x + sum.y, red[0]) * inv : 0.0f;
        float2 sq = splat2(0.0f);
#pragma unroll
        for (int j = 0; j < VPT; j++)
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                float2 v = add2(pair(u[j], e), splat2(-mean));
                if (!on[j]) v = splat2(0.0f);
                if (E == 1) v.y = 0.0f;
                sq = fma2(v, v, sq);
                put(u[j], e, v);
            }
        const float var = group_sum<LPG>(sq.x + sq.y, red[1]) * inv;
        // (a warp beyond the last row: with eps = 0 its 0 * inf would reach the parameters' sums)
        const float rstd = !BWD || LPG == 0 || row ? rsqrtf(var + a.eps) : 0.0f;
        if (!BWD) {
#pragma unroll
            for (int j = 0; j < VPT; j++) {
                float o[E];
                if (VPT > 1) params(j, w[0], bb[0]);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 n = fma2(mul2(pair(u[j], e), splat2(rstd)), pair(w[0], e), pair(bb[0], e));
                    const float2 zv = gate ? pair(z[j], e) : n;
                    put(o, e, gate && first ? n : mul2(n, gate ? mul2(zv, sigmoid(zv)) : sigmoid(zv)));
                }
                if (row && on[j]) store<T, E>(a.out, at + (int64_t)(l + j * lanes) * E, o);
            }
        } else {
            float2 s1 = splat2(0.0f), s2 = splat2(0.0f);  // sums of t and t * xhat, t the gradient of xhat
#pragma unroll
            for (int j = 0; j < VPT; j++) {
                float o[E];
                if (VPT > 1) params(j, w[0], bb[0]);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 xh = mul2(pair(u[j], e), splat2(rstd)), wv = pair(w[0], e);
                    const float2 n = fma2(xh, wv, pair(bb[0], e));
                    float2 g = pair(d[j], e);
                    if (!(gate && first)) {
                        const float2 v = gate ? pair(z[j], e) : n, sg = sigmoid(v), f = mul2(v, sg);
                        // silu'(v) = sg (1 + v (1 - sg)) = sg + f - f sg
                        const float2 df = fma2(f, fma2(sg, splat2(-1.0f), splat2(1.0f)), sg);
                        if (gate) {
                            put(o, e, mul2(mul2(g, n), df));
                            g = mul2(g, f);
                        } else {
                            g = mul2(g, df);
                        }
                    }
                    put(dw[j], e, fma2(g, xh, pair(dw[j], e)));
                    put(db[j], e, add2(g, pair(db[j], e)));
                    const float2 t = mul2(g, wv);
                    s1 = add2(s1, t);
                    s2 = fma2(t, xh, s2);
                    put(d[j], e, t);
                    put(u[j], e, xh);
                }
                if (gate && !first && row && on[j]) store<T, E>(a.dz, at + (int64_t)(l + j * lanes) * E, o);
            }
            const float2 m = group_sum2<LPG>(E > 1 ? make_float2(s1.x + s1.y, s2.x + s2.y) : make_float2(s1.x, s2.x), red[2], red[3]);
            const float m1 = center ? m.x * inv : 0.0f, m2 = m.y * inv;
#pragma unroll
            for (int j = 0; j < VPT; j++) {
                float o[E], o2[E];
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    float2 du = fma2(pair(u[j], e), splat2(-m2), add2(pair(d[j], e), splat2(-m1)));
                    du = mul2(du, splat2(rstd));
                    if (gate && first) {
                        const float2 v = pair(z[j], e), sg = sigmoid(v), f = mul2(v, sg);
                        const float2 df = fma2(f, fma2(sg, splat2(-1.0f), splat2(1.0f)), sg);
                        put(o2, e, mul2(mul2(du, pair(x[j], e)), df));
                        du = mul2(du, f);
                    }
                    put(o, e, du);
                }
                const int64_t i = at + (int64_t)(l + j * lanes) * E;
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
            if (LPG > 0) {
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
                    const int64_t c = grp * gs + (int64_t)(l + j * lanes) * E;
#pragma unroll
                    for (int e = 0; e < E; e++) {
                        float v = pass ? db[j][e] : dw[j][e];
                        if (LPG > 0) {
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

// Row blocks of a launch, xblocks blocks wide, of which per_sm fit on an SM: one
// round of blocks, each walking over its share of the rows.
int64_t row_blocks(int64_t M, int64_t xblocks, int64_t rows, int64_t per_sm) {
    const int64_t want = la::kSms * per_sm / xblocks, most = ceil_div(M, rows);
    const int64_t y = want < most ? want : most;
    return y < 1 ? 1 : (y > 65535 ? 65535 : y);
}

template <typename T, int E, int LPG, int VPT, bool BWD> cudaError_t go(const GnormArgs& a, cudaStream_t st) {
    const int64_t x = LPG > 0 ? ceil_div(a.groups * LPG, 32) : a.groups;
    // the block that covers a group: whole warps, no more than its runs need
    const int threads = LPG > 0 ? 256 : (int)(ceil_div(ceil_div(a.C / a.groups / E, VPT), 32) * 32);
    const int64_t y = BWD ? gnorm_bwd_blocks(a.M, a.C, a.groups)
                          : row_blocks(a.M, x, kRowsPerStep<LPG>, LPG > 0 ? kPerSm<LPG, VPT, BWD> : ceil_div(1280, threads));
    constexpr int slot = kRing<E> ? kDepth<LPG, VPT, BWD> * (BWD ? 3 : 2) * VPT * 16 : 0;  // bytes a thread
    const int smem = slot * threads;
    const cudaError_t e = la::allow_smem<k_gnorm<T, E, LPG, VPT, BWD>>(slot * (LPG > 0 ? 256 : (VPT <= 2 ? 640 : 512)));
    if (e != cudaSuccess) return e;
    k_gnorm<T, E, LPG, VPT, BWD><<<dim3((unsigned)x, (unsigned)y), threads, smem, st>>>(a);
    return cudaGetLastError();
}

bool aligned(const GnormArgs& a) {
    const void* p[] = {a.x, a.z, a.dout, a.out, a.dx, a.dz, a.weight, a.bias};
    for (const void* q : p)
        if (reinterpret_cast<uintptr_t>(q) & 15u) return false;
    return true;
}

// The threads that hold a group, by the number of 16-byte runs in it: part of a warp, a
// warp with up to four runs a lane (groups of 1024: 109 and 144 us, with a block each
// 119 and 361), then a block.  Groups that are no whole number of runs, and unaligned
// tensors, move value by value (groups of 64 would take 909 and 1281 us that way).
template <typename T, bool BWD> cudaError_t pick(const GnormArgs& a, cudaStream_t st) {
    constexpr int E = 16 / (int)sizeof(T);
    const int64_t gs = a.C / a.groups;
    if (gs % E != 0 || !aligned(a)) {
        if (gs <= 256) return go<T, 1, 32, 8, BWD>(a, st);
        if (gs <= 2048) return go<T, 1, 0, 4, BWD>(a, st);
        return go<T, 1, 0, 16, BWD>(a, st);
    }
    const int64_t n = gs / E;
    if (n <= 4) return go<T, E, 4, 1, BWD>(a, st);
    if (n <= 8) return go<T, E, 8, 1, BWD>(a, st);
    if (n <= 16) return go<T, E, 16, 1, BWD>(a, st);
    if (n <= 32) return go<T, E, 32, 1, BWD>(a, st);
    if (n <= 64) return go<T, E, 32, 2, BWD>(a, st);
    if (n <= 128) return go<T, E, 32, 4, BWD>(a, st);
    if (n <= 640) return go<T, E, 0, 1, BWD>(a, st);
    // (8192 channels are at most 1024 runs of 16-bit values, 2048 of f32)
    if constexpr (E == 4)
        if (n > 1280) return go<T, E, 0, 4, BWD>(a, st);
    return go<T, E, 0, 2, BWD>(a, st);
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
    if (gs > 1024) return row_blocks(M, groups, 1, ceil_div(5120, gs));
    return row_blocks(M, gs > 256 ? groups : ceil_div(C, 256), 8, gs > 256 ? 1 : 2);
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
