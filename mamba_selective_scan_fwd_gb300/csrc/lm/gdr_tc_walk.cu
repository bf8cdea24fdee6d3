// Gated delta rule on the tensor cores: the walk over the chunks.
//
// One block walks the chunks of one segment of one (batch row, head, 128 value channels)
// with the state transposed: the value channels are the 128 lanes of tensor memory, so that
// a thread owns a channel (half of its N states, half of a chunk's tokens) and every
// left operand is written by the thread that will read the product's row:
//   D1 = S^T K^T             [128 x 64]   S in two 16-bit parts, from tensor memory
//   X = beta (V^T - e^c D1)               two bf16 parts
//   D2 = X M^T = U^T         [128 x 64]   lo hi + hi lo + hi hi
//   D3 = (e^{cl - c} U)^T K  [128 x N]    two 16-bit parts;  S <- e^{cl} S + D3, f32 in registers
//   y = scale (e^c S^T Q^T + U^T P^T)     off the chain: a third warpgroup writes it
// A loading warp copies a chunk's tiles one chunk ahead and issues all products.  Chain of a
// chunk: three products and three passes through the registers.
//
// Roundings: two 16-bit parts of S, X, M and e U hold 16 bits (f16: 22) of each, which leaves
// the f32 state good to a few 1e-6; P and U enter y's product with one bf16 part each (f16 io:
// two), one rounding each of terms of a 16-bit y.  f16's S and e U are scaled by a power of two
// per channel, taken from their largest value.
#include "gdr_tc.h"
#include "../simd.cuh"
#include "tc.cuh"
#include "gdr_dev.cuh"

namespace ss {
namespace gdr {
namespace {

using la::kF16;
using la::pack2;
using la::unit;
using la::unpack2;
using la::wait_or_fail;
using bf16 = __nv_bfloat16;

constexpr int C = kChunk;
constexpr int kStateThreads = 256, kThreads = 256 + 128 + 32;

// columns of tensor memory: D1 then D2; S^T Q^T; D3; U^T P^T; parts of S, then of e U; parts of X, then of U
constexpr uint32_t kD1 = 0, kQ = 64, kD3 = 128, kY = 256, kS = 320, kX = 448;

template <typename T> constexpr int kPParts = kF16<T> ? 2 : 1;

template <typename T, int NB> struct Stage {
    static constexpr int k = 0, q = k + NB * kTileBytes, v = q + NB * kTileBytes, image = v + 2 * kTileBytes,
                         head = image + (2 + kPParts<T>) * kTileBytes, bytes = head + 1024;
};

__device__ __forceinline__ void arrive(uint64_t* bar) {  // a warp's
    la::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) la::mbar_arrive(bar);
}
__device__ __forceinline__ void named_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// 32 values as two 16-bit parts: 16 columns of tensor memory each
template <typename T> __device__ __forceinline__ void put2(uint32_t hi, uint32_t lo, const float (&x)[32], float s) {
    uint32_t r[16], q[16];
#pragma unroll
    for (int i = 0; i < 16; i++) {
        float2 f = make_float2(x[2 * i], x[2 * i + 1]);
        if (kF16<T>) f = mul2(f, splat2(s));
        r[i] = pack2<T>(f.x, f.y);
        f = fma2(unpack2<T>(r[i]), splat2(-1.0f), f);
        q[i] = pack2<T>(f.x, f.y);
    }
    la::tmem_st16(hi, r);
    la::tmem_st16(lo, q);
}
template <typename T> __device__ __forceinline__ void put1(uint32_t to, const float (&x)[32]) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; i++) r[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
    la::tmem_st16(to, r);
}

// SUM: no y.  blockIdx.y of SUM: 0 walks from zero (E), 1 from the identity without v (Phi).
template <typename T, int NB, bool SUM>
__global__ void __launch_bounds__(kThreads, 1) k_walk(const __grid_constant__ TcWalkArgs w) {
    extern __shared__ __align__(1024) char sm[];
    using L = Stage<T, NB>;
    constexpr int W = 32 * NB;  // states of a thread
    constexpr int PP = kPParts<T>;
    __shared__ __align__(8) uint64_t s_full[2], s_s, s_d1, s_x, s_d2, s_u, s_d3, s_y, s_done;
    __shared__ uint32_t s_tm, s_fail;
    __shared__ float s_max[2][2][128], s_ss[2][128];
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pl = tid & 127;
    const bool phi = SUM && blockIdx.y == 1;
    const int64_t width = phi ? a.N : a.P, ptiles = (width + kTileP - 1) / kTileP;
    int64_t id = blockIdx.x;
    // phi has fewer tiles of columns than v may have: the blocks beyond do nothing
    const int64_t p0 = id % ((a.P + kTileP - 1) / kTileP) * kTileP;
    id /= (a.P + kTileP - 1) / kTileP;
    if (phi && p0 >= ptiles * kTileP) return;
    const int64_t bh = id % (a.Bsz * a.H), seg = id / (a.Bsz * a.H);
    const int64_t b = bh / a.H, h = bh % a.H, hq = h / (a.H / a.G);
    const int64_t len = row_length(a, b);
    const int64_t c_begin = seg * w.plan.seg, t_begin = c_begin * C, t_end = min(a.L, (c_begin + w.plan.seg) * C);
    const int chunks = (int)max((int64_t)0, (min(len, t_end) - t_begin + C - 1) / C);

    if (tid == 0) {
        for (uint64_t* bar : {&s_full[0], &s_full[1], &s_d1, &s_d2, &s_d3, &s_y}) mbar_init(bar, 1);
        for (uint64_t* bar : {&s_s, &s_x, &s_u}) mbar_init(bar, kStateThreads / 32);
        mbar_init(&s_done, 4);
        s_fail = 0;
        fence_proxy_async_smem();
    }
    if (warp == 0) la::tmem_alloc(&s_tm, 512);
    __syncthreads();
    la::tc_fence_after();
    const uint32_t tm = s_tm, my = (uint32_t)((warp & 3) * 32) << 16;
    char* Y = sm + 2 * L::bytes;  // staging of y: two tiles of [token][64 channels]
    auto valid = [&](int ch) { return (int)min((int64_t)C, len - (t_begin + (int64_t)ch * C)); };

    if (warp < kStateThreads / 32) {
        const int half = tid >> 7;
        const int64_t p = p0 + pl;
        const bool mine = p < width;
        float S[W];
        if (phi) {
#pragma unroll
            for (int n = 0; n < W; n++) S[n] = half * W + n == p ? 1.0f : 0.0f;
        } else {
            const float* from = SUM ? nullptr : w.plan.K > 1 ? w.seg_state + (bh * w.plan.K + seg) * a.N * a.P
                                                             : (w.init ? w.init + bh * a.N * a.P : nullptr);
#pragma unroll
            for (int n = 0; n < W; n++) S[n] = from && mine && half * W + n < a.N ? from[(half * W + n) * a.P + p] : 0.0f;
        }
        // (a wait that ran out ends no loop here: the others wait at its barriers)
        // f16: the power of two of this channel's row, from both halves' largest values
        auto row_scale = [&](float most, int which) {
            s_max[which][half][pl] = most;
            named_sync(1, kStateThreads);
            return la::f16_scale(fmaxf(s_max[which][0][pl], s_max[which][1][pl]));
        };
        bool ok = true;
        for (int ch = 0; ch < chunks; ch++) {
            const uint32_t ph = ch & 1;
            char* at = sm + ph * L::bytes;
            const ImageHead* head = reinterpret_cast<const ImageHead*>(at + L::head);
            const int nv = valid(ch);
            float ss = 1.0f;
            if (kF16<T>) {
                float m = 0.0f;
#pragma unroll
                for (int n = 0; n < W; n++) m = fmaxf(m, fabsf(S[n]));
                ss = row_scale(m, 0);
                if (half == 0) s_ss[ph][pl] = ss;  // y's product has it too
            }
#pragma unroll
            for (int c = 0; c < NB; c++) {
                float x[32];
#pragma unroll
                for (int n = 0; n < 32; n++) x[n] = S[32 * c + n];
                const uint32_t to = tm + my + kS + half * (W / 2) + 16 * c;
                put2<T>(to, to + 32 * NB, x, ss);
            }
            la::tmem_wait_st();
            ok = ok && wait_or_fail(&s_full[ph], (ch >> 1) & 1, &s_fail);
            if (nv < C && ok) {  // keys past the row's length: zero, whatever they hold
                const int row = tid & 63;
                if (row >= nv && (tid >> 6) < NB)
#pragma unroll
                    for (int u = 0; u < 8; u++) *unit(at + L::k + (tid >> 6) * kTileBytes, row, u) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            arrive(&s_s);
            float vv[32];
            {
                const char* tile = at + L::v + (pl >> 6) * kTileBytes;
                const int c = (pl & 63) >> 3, e = (pl & 7) * 2;
#pragma unroll
                for (int j = 0; j < 32; j++) {
                    const int t = 32 * half + j;
                    vv[j] = phi ? 0.0f : ldf(reinterpret_cast<const T*>(tile + t * 128 + ((c ^ (t & 7)) << 4) + e));
                }
            }
            ok = ok && wait_or_fail(&s_d1, ph, &s_fail);
            la::tc_fence_after();
            float d[32];
            la::tmem_ld32(tm + my + kD1 + 32 * half, d);
            const float inv = kF16<T> ? 1.0f / ss : 1.0f;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 up = *reinterpret_cast<const float4*>(&head->up[32 * half + j]);
                const float4 be = *reinterpret_cast<const float4*>(&head->beta[32 * half + j]);
                const float us[4] = {up.x, up.y, up.z, up.w}, bs[4] = {be.x, be.y, be.z, be.w};
#pragma unroll
                for (int e = 0; e < 4; e++) d[j + e] = bs[e] * fmaf(-(kF16<T> ? us[e] * inv : us[e]), d[j + e], vv[j + e]);
            }
            if (nv < C) {
#pragma unroll
                for (int j = 0; j < 32; j++)
                    if (32 * half + j >= nv) d[j] = 0.0f;
            }
            {
                const uint32_t to = tm + my + kX + 16 * half;
                put2<bf16>(to, to + 32, d, 1.0f);
            }
            la::tmem_wait_st();
            arrive(&s_x);
            ok = ok && wait_or_fail(&s_d2, ph, &s_fail);
            la::tc_fence_after();
            la::tmem_ld32(tm + my + kD1 + 32 * half, d);
            if (!SUM) {
                const uint32_t to = tm + my + kX + 16 * half;
                if (PP > 1) put2<bf16>(to, to + 32, d, 1.0f);
                else put1<bf16>(to, d);
            }
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&head->down[32 * half + j]);
                d[j] *= f.x;
                d[j + 1] *= f.y;
                d[j + 2] *= f.z;
                d[j + 3] *= f.w;
            }
            float us = 1.0f;
            if (kF16<T>) {
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < 32; j++) m = fmaxf(m, fabsf(d[j]));
                us = row_scale(m, 1);
            }
            {
                const uint32_t to = tm + my + kS + 16 * half;
                put2<T>(to, to + 32, d, us);
            }
            la::tmem_wait_st();
            const la::Decay by = {head->by, head->weak != 0};
            arrive(&s_u);
            ok = ok && wait_or_fail(&s_d3, ph, &s_fail);
            la::tc_fence_after();
            const float uinv = kF16<T> ? 1.0f / us : 1.0f;
#pragma unroll
            for (int c = 0; c < NB; c++) {
                la::tmem_ld32(tm + my + kD3 + half * W + 32 * c, d);
#pragma unroll
                for (int n = 0; n < 32; n++) S[32 * c + n] = fmaf(uinv, d[n], la::decayed(by, S[32 * c + n]));
            }
            if (!ok) break;
        }
        if (mine && !s_fail) {
            float* to = nullptr;
            if (phi) to = w.seg_phi + (bh * w.plan.K + seg) * a.N * a.N;
            else if (SUM) to = w.seg_state + (bh * w.plan.K + seg) * a.N * a.P;
            else if (seg == w.plan.K - 1 && w.last) to = w.last + bh * a.N * a.P;
            if (to)
#pragma unroll
                for (int n = 0; n < W; n++)
                    if (half * W + n < a.N) to[(half * W + n) * width + p] = S[n];
        }
    } else if (warp < kStateThreads / 32 + 4) {
        if (!SUM) {
            T* yp = static_cast<T*>(w.yp) + (b * a.L * a.H + h) * a.P;
            const bool wide = p0 + 64 < a.P;
            for (int ch = 0; ch < chunks; ch++) {
                const uint32_t ph = ch & 1;
                const ImageHead* head = reinterpret_cast<const ImageHead*>(sm + ph * L::bytes + L::head);
                const int nv = valid(ch);
                if (tid == kStateThreads) la::bulk_wait_read();
                named_sync(2, 128);  // the staging tiles are free
                wait_or_fail(&s_full[ph], (ch >> 1) & 1, &s_fail);
                wait_or_fail(&s_y, ph, &s_fail);
                la::tc_fence_after();
                const float inv = kF16<T> ? a.scale / s_ss[ph][pl] : a.scale;
                char* tile = Y + (pl >> 6) * kTileBytes;
                const int cu = (pl & 63) >> 3, eb = (pl & 7) * 2;
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    float q[32], y[32];
                    la::tmem_ld32(tm + my + kQ + 32 * hf, q);
                    la::tmem_ld32(tm + my + kY + 32 * hf, y);
#pragma unroll
                    for (int j = 0; j < 32; j++) {
                        const int t = 32 * hf + j;
                        const float x = fmaf(inv * head->up[t], q[j], a.scale * y[j]);
                        st(reinterpret_cast<T*>(tile + t * 128 + ((cu ^ (t & 7)) << 4) + eb), t < nv ? x : 0.0f);
                    }
                }
                arrive(&s_done);
                fence_proxy_async_smem();
                named_sync(2, 128);
                if (tid == kStateThreads) {
                    const int64_t t0 = t_begin + (int64_t)ch * C;
                    la::tma_store_4d(&w.y, Y, (int)p0, (int)h, (int)t0, (int)b);
                    if (wide) la::tma_store_4d(&w.y, Y + kTileBytes, (int)p0 + 64, (int)h, (int)t0, (int)b);
                    la::bulk_commit();
                }
            }
            if (tid == kStateThreads) la::bulk_wait_all();
            // tokens of chunks beyond the row's length
            for (int64_t t = t_begin + (int64_t)chunks * C + (warp & 3); t < t_end; t += 4)
                for (int64_t p = p0 + lane * 8; p < min(a.P, p0 + kTileP); p += 256)
                    *reinterpret_cast<uint4*>(yp + t * a.H * a.P + p) = make_uint4(0, 0, 0, 0);
        }
    } else if (lane == 0) {
        auto load = [&](int ch) {
            char* at = sm + (ch & 1) * L::bytes;
            uint64_t* bar = &s_full[ch & 1];
            const int t0 = (int)(t_begin + (int64_t)ch * C);
            mbar_expect_tx(bar, ((SUM ? 1 : 2) * NB + (phi ? 0 : 2)) * kTileBytes + image_bytes(PP));
#pragma unroll
            for (int n = 0; n < NB; n++) {
                la::tma_load_4d(at + L::k + n * kTileBytes, &w.k, n * 64, (int)hq, t0, (int)b, bar);
                if (!SUM) la::tma_load_4d(at + L::q + n * kTileBytes, &w.q, n * 64, (int)hq, t0, (int)b, bar);
            }
            if (!phi) {
                la::tma_load_4d(at + L::v, &w.v, (int)p0, (int)h, t0, (int)b, bar);
                la::tma_load_4d(at + L::v + kTileBytes, &w.v, (int)p0 + 64, (int)h, t0, (int)b, bar);
            }
            bulk_load(at + L::image, w.images + (bh * w.chunks + c_begin + ch) * image_bytes(PP), image_bytes(PP), bar);
        };
        if (chunks > 0) load(0);
        if (chunks > 1) load(1);
        for (int ch = 0; ch < chunks; ch++) {
            const uint32_t ph = ch & 1;
            const uint32_t at = smem_addr(sm + ph * L::bytes), K = at + L::k, Q = at + L::q, M = at + L::image,
                           P = M + 2 * kTileBytes;
            constexpr uint32_t dK = la::mma_desc<T>(128, C, false, false), dM = la::mma_desc<bf16>(128, C, false, false),
                               dU = la::mma_desc<T>(128, 64 * NB, false, true);
            if (!wait_or_fail(&s_full[ph], (ch >> 1) & 1, &s_fail) || !wait_or_fail(&s_s, ph, &s_fail)) break;
            la::tc_fence_after();
            auto with_state = [&](uint32_t to, uint32_t tile, int parts) {
                for (int part = parts - 1; part >= 0; part--)
#pragma unroll
                    for (int s = 0; s < 4 * NB; s++)
                        la::mma_ts(tm + to, tm + kS + part * 32 * NB + 8 * s, la::smem_desc(tile + (s >> 2) * kTileBytes + (s & 3) * 32), dK,
                                   part < parts - 1 || s > 0);
            };
            with_state(kD1, K, 2);
            la::mma_commit(&s_d1);
            if (!SUM) {
                // y of the chunk before is out of tensor memory, and with it all products of that chunk are done
                if (ch > 0 && !wait_or_fail(&s_done, ph ^ 1, &s_fail)) break;
                with_state(kQ, Q, PP);
            }
            if (ch > 0 && ch + 1 < chunks) load(ch + 1);
            if (!wait_or_fail(&s_x, ph, &s_fail)) break;
            la::tc_fence_after();
            auto parts_by = [&](uint32_t to, uint32_t left, uint32_t tile, bool wide) {  // 64 tokens; lo hi + hi lo + hi hi
#pragma unroll
                for (int o = wide ? 0 : 2; o < 3; o++)
#pragma unroll
                    for (int s = 0; s < 4; s++)
                        la::mma_ts(tm + to, tm + left + (o == 0 ? 32 : 0) + 8 * s, la::smem_desc(tile + (o == 1 ? kTileBytes : 0) + s * 32), dM,
                                   o > (wide ? 0 : 2) || s > 0);
            };
            parts_by(kD1, kX, M, true);
            la::mma_commit(&s_d2);
            if (!wait_or_fail(&s_u, ph, &s_fail)) break;
            la::tc_fence_after();
#pragma unroll
            for (int part = 1; part >= 0; part--)
#pragma unroll
                for (int s = 0; s < 4; s++)
                    la::mma_ts(tm + kD3, tm + kS + part * 32 + 8 * s, la::smem_desc(K + s * 2048, kTileBytes), dU, part < 1 || s > 0);
            la::mma_commit(&s_d3);
            if (!SUM) {
                parts_by(kY, kX, P, PP > 1);
                la::mma_commit(&s_y);
            }
        }
    }
    __syncwarp();
    uint64_t* const bars[6] = {&s_full[0], &s_full[1], &s_d1, &s_d2, &s_d3, &s_y};
    la::end_block(&s_fail, w.status, bars, tm, 512);
}

// S <- Phi S + E over the segments, from h0; seg_state receives the state each segment starts
// from.  A block: 16 columns of one head's state, kept in shared memory.
__global__ void __launch_bounds__(256) k_carry(TcWalkArgs w) {
    constexpr int NC = 16;
    __shared__ float s[2][la::kMaxN][NC];
    const Args& a = w.a;
    const int tid = threadIdx.x, N = (int)a.N;
    const int64_t ptiles = (a.P + NC - 1) / NC, p0 = blockIdx.x % ptiles * NC, bh = blockIdx.x / ptiles;
    const int c = tid % NC, r = tid / NC;
    const bool mine = p0 + c < a.P;
    float own[la::kMaxN / 16];
#pragma unroll
    for (int u = 0; u < la::kMaxN / 16; u++) {
        const int n = r + 16 * u;
        s[0][n][c] = mine && n < N && w.init ? w.init[(bh * N + n) * a.P + p0 + c] : 0.0f;
    }
    for (int64_t k = 0; k < w.plan.K; k++) {
        float* at = w.seg_state + (bh * w.plan.K + k) * N * a.P + p0 + c;
        const float* phi = w.seg_phi + (bh * w.plan.K + k) * N * N;
        float(*now)[NC] = s[k & 1], (*next)[NC] = s[~k & 1];
#pragma unroll
        for (int u = 0; u < la::kMaxN / 16; u++) {
            const int n = r + 16 * u;
            own[u] = mine && n < N && k + 1 < w.plan.K ? at[n * a.P] : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < la::kMaxN / 16; u++) {
            const int n = r + 16 * u;
            if (mine && n < N) at[n * a.P] = now[n][c];
        }
        if (k + 1 == w.plan.K) break;
#pragma unroll 2
        for (int m = 0; m < N; m += 4) {
            const float x[4] = {now[m][c], now[m + 1][c], now[m + 2][c], now[m + 3][c]};
#pragma unroll
            for (int u = 0; u < la::kMaxN / 16; u++) {
                const int n = r + 16 * u;
                if (n >= N) continue;
                const float4 f = *reinterpret_cast<const float4*>(phi + n * N + m);
                own[u] = fmaf(f.x, x[0], fmaf(f.y, x[1], fmaf(f.z, x[2], fmaf(f.w, x[3], own[u]))));
            }
        }
#pragma unroll
        for (int u = 0; u < la::kMaxN / 16; u++) next[r + 16 * u][c] = own[u];
    }
}

template <typename T, int NB, bool SUM> cudaError_t walk_go(const TcWalkArgs& w, cudaStream_t st) {
    constexpr int bytes = 2 * Stage<T, NB>::bytes + (SUM ? 0 : 2 * kTileBytes);
    const cudaError_t e = la::allow_smem<k_walk<T, NB, SUM>>(bytes);
    if (e != cudaSuccess) return e;
    const int64_t segs = SUM ? w.plan.K - 1 : w.plan.K;
    const dim3 grid((unsigned)(ceil_div(w.a.P, kTileP) * w.a.Bsz * w.a.H * segs), SUM ? 2 : 1);
    k_walk<T, NB, SUM><<<grid, kThreads, bytes, st>>>(w);
    return cudaGetLastError();
}
template <typename T, int NB> cudaError_t walk_mode(const TcWalkArgs& w, TcWalkMode mode, cudaStream_t st) {
    return mode == kTcSum ? walk_go<T, NB, true>(w, st) : walk_go<T, NB, false>(w, st);
}

}  // namespace

cudaError_t launch_tc_walk(const TcWalkArgs& w, TcWalkMode mode, cudaStream_t st) {
    if (w.a.dtype == 1) return w.a.N <= 64 ? walk_mode<__half, 1>(w, mode, st) : walk_mode<__half, 2>(w, mode, st);
    return w.a.N <= 64 ? walk_mode<bf16, 1>(w, mode, st) : walk_mode<bf16, 2>(w, mode, st);
}

cudaError_t launch_tc_carry(const TcWalkArgs& w, cudaStream_t st) {
    k_carry<<<(unsigned)(ceil_div(w.a.P, 16) * w.a.Bsz * w.a.H), 256, 0, st>>>(w);
    return cudaGetLastError();
}

}  // namespace gdr
}  // namespace ss
