// Linear attention on the tensor cores: the forward, and the states at the
// chunks' borders that the backward reads.  16-bit io.
//
// A chunk is 128 tokens (the M of a matrix product).  With c_i the cumulative
// log decay inside the chunk, cl its end and H the state before it:
//   S = q k^T,  P_ij = e^{c_i - c_j} S_ij (j <= i),  y = scale (e^{c_i} q H + P v)
//   H <- e^{cl} H + k^T (e^{cl - c} v)
// One block walks one segment of one (batch row, head, 64 value channels) and
// keeps H in f32 registers (thread = one of the N rows): S, q H and k^T (w v)
// are products of tiles that TMA brought, P is the left operand out of tensor
// memory.  Roundings to 16 bits: P, and H as an operand of q H (one rounding of
// terms of a 16-bit y each).  The state is f32: w v enters as two or three
// 16-bit parts whose sum holds 22 to 24 bits.
#include "la_tc.h"
#include "tc.cuh"

namespace ss {
namespace la {
namespace {

constexpr int C = kChunkTc;
constexpr int PT = kTileP;

template <typename T> constexpr bool kF16 = false;
template <> constexpr bool kF16<__half> = true;
// 16-bit parts of w v: 3 x 8 bits (bf16), 2 x 11 (f16)
template <typename T> constexpr int kParts = kF16<T> ? 2 : 3;

// The chunk's decays, by runs of 32 tokens (one warp's).  c_i = (the run's end)
// - rel_i; rel is a thread's own, the rest is shared.
struct Decays {
    float tail[C];  // e^{rel}
    Two total[4];   // log2 decay of each run
};

// Both halves of the block (256 threads, token = tid % 128), x: the token's log2
// decay.  Returns rel (at most 0 for decays).
__device__ __forceinline__ float chunk_decays(Decays& d, float x) {
    const float in[1] = {x};
    Two c[1];
    warp_cumsum<1>(in, c);
    const Two end = {__shfl_sync(kFull, c[0].h, 31), __shfl_sync(kFull, c[0].l, 31)};
    const float rel = two_diff(end, c[0]);
    if (threadIdx.x < C) {
        d.tail[threadIdx.x] = ex2(rel);
        if ((threadIdx.x & 31) == 31) d.total[threadIdx.x >> 5] = end;
    }
    return rel;
}
// After a barrier: log2 decays from the chunk's start to the end of each run.
__device__ __forceinline__ void run_ends(const Decays& d, Two (&end)[4]) {
    end[0] = d.total[0];
#pragma unroll
    for (int i = 1; i < 4; i++) end[i] = two_add(end[i - 1], d.total[i]);
}
__device__ __forceinline__ float load_g(const Args& a, int64_t b, int64_t h, int64_t t0, int nv) {
    const int t = threadIdx.x & (C - 1);
    return t < nv ? log_decay(a, b, t0 + t, h) * kLog2e : 0.0f;
}

// Largest value of the block's threads (all get it); v >= 0.  Two block barriers.
__device__ __forceinline__ float block_max(float v, uint32_t* red) {
    uint32_t m;
    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(__float_as_uint(v)));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = max(max(max(red[0], red[1]), max(red[2], red[3])), max(max(red[4], red[5]), max(red[6], red[7])));
    __syncthreads();
    return __uint_as_float(m);
}

// Half of row `row` of a value tile, times w, as 16-bit parts (same layout).
template <typename T> __device__ __forceinline__ void split_row(void* v, int row, int half, float w, void* p0, void* p1, void* p2) {
#pragma unroll 2
    for (int u = 4 * half; u < 4 * half + 4; u++) {
        const uint4 in = *unit(v, row, u);
        const uint32_t x[4] = {in.x, in.y, in.z, in.w};
        uint32_t r[3][4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float2 f = unpack2<T>(x[i]);
            f.x *= w;
            f.y *= w;
#pragma unroll
            for (int k = 0; k < kParts<T>; k++) {
                r[k][i] = pack2<T>(f.x, f.y);
                const float2 g = unpack2<T>(r[k][i]);
                f.x -= g.x;
                f.y -= g.y;
            }
        }
        *unit(p0, row, u) = make_uint4(r[0][0], r[0][1], r[0][2], r[0][3]);
        *unit(p1, row, u) = make_uint4(r[1][0], r[1][1], r[1][2], r[1][3]);
        if (kParts<T> == 3) *unit(p2, row, u) = make_uint4(r[2][0], r[2][1], r[2][2], r[2][3]);
    }
}

template <typename T> __device__ __forceinline__ float row_max(void* v, int row, int half) {
    float m = 0.0f;
#pragma unroll
    for (int u = 4 * half; u < 4 * half + 4; u++) {
        const uint4 in = *unit(v, row, u);
        const uint32_t x[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = unpack2<T>(x[i]);
            m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
    }
    return m;
}

// The state a thread of 256 holds: NB == 2, row tid % 128, 32 of the 64 columns;
// NB == 1, row tid % 64, 16 columns (the product's 128 rows hold the 64 twice).
template <int NB> struct StateOf {
    static constexpr int W = 16 * NB;
    __device__ static int row() { return threadIdx.x & (64 * NB - 1); }
    __device__ static int col() { return (int)(threadIdx.x / (64 * NB)) * W; }
};

template <int NB> __device__ __forceinline__ void load_state(const float* p, const Args& a, int64_t p0, float (&X)[16 * NB]) {
    const int n = StateOf<NB>::row(), c0 = StateOf<NB>::col();
#pragma unroll
    for (int c = 0; c < 16 * NB; c += 4) {
        float4 f = {0.0f, 0.0f, 0.0f, 0.0f};
        if (p && n < a.N && p0 + c0 + c < a.P) f = *reinterpret_cast<const float4*>(p + n * a.P + p0 + c0 + c);
        X[c] = f.x;
        X[c + 1] = f.y;
        X[c + 2] = f.z;
        X[c + 3] = f.w;
    }
}
template <int NB> __device__ __forceinline__ void save_state(float* p, const Args& a, int64_t p0, const float (&X)[16 * NB]) {
    const int n = StateOf<NB>::row(), c0 = StateOf<NB>::col();
#pragma unroll
    for (int c = 0; c < 16 * NB; c += 4)
        if (n < a.N && p0 + c0 + c < a.P)
            *reinterpret_cast<float4*>(p + n * a.P + p0 + c0 + c) = make_float4(X[c], X[c + 1], X[c + 2], X[c + 3]);
}
template <int NB> __device__ __forceinline__ float state_max(const float (&X)[16 * NB]) {
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < 16 * NB; c++) m = fmaxf(m, fabsf(X[c]));
    return m;
}
__device__ __forceinline__ void tmem_ldw(uint32_t addr, float (&x)[16]) { tmem_ld16(addr, x); }
__device__ __forceinline__ void tmem_ldw(uint32_t addr, float (&x)[32]) { tmem_ld32(addr, x); }
// X <- d X + u * (the product in tensor memory)
template <int NB> __device__ __forceinline__ void add_product(uint32_t tm, float d, float u, float (&X)[16 * NB]) {
    float f[16 * NB];
    tmem_ldw(tm + ((threadIdx.x & 96) << 16) + StateOf<NB>::col(), f);
#pragma unroll
    for (int i = 0; i < 16 * NB; i++) X[i] = fmaf(d, X[i], u * f[i]);
}
// 16-bit rows [n][p] of X * s (and of what the rounding left): operand tiles
template <typename T, int NB> __device__ __forceinline__ void put_state(void* hi, void* lo, float s, const float (&X)[16 * NB]) {
    const int n = StateOf<NB>::row(), u0 = StateOf<NB>::col() / 8;
#pragma unroll
    for (int u = 0; u < 2 * NB; u++) {
        uint32_t r[4], q[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float x = X[8 * u + 2 * i] * s, y = X[8 * u + 2 * i + 1] * s;
            r[i] = pack2<T>(x, y);
            const float2 g = unpack2<T>(r[i]);
            q[i] = pack2<T>(x - g.x, y - g.y);
        }
        *unit(hi, n, u0 + u) = make_uint4(r[0], r[1], r[2], r[3]);
        if (lo) *unit(lo, n, u0 + u) = make_uint4(q[0], q[1], q[2], q[3]);
    }
}

// k^T (w v): rows n (both halves of the 128 rows the same 64 when NB == 1), columns p
template <typename T, int NB> __device__ __forceinline__ void mma_state(uint32_t tm, const void* k, const void* const (&w)[3]) {
    constexpr uint32_t desc = mma_desc<T>(128, PT, true, true);
    const uint32_t ka = smem_addr(k);
#pragma unroll
    for (int p = 0; p < kParts<T>; p++)
#pragma unroll
        for (int s = 0; s < C / 16; s++)
            mma(tm, smem_desc(ka + s * 2048, NB == 2 ? 16384 : 0), smem_desc(smem_addr(w[p]) + s * 2048), desc, p + s > 0);
}

// Half a row of each tile that a copy filled with a token beyond the row's length: zero.
template <int TILES> __device__ __forceinline__ void clear_row(char* const (&tiles)[TILES], int row, int half) {
#pragma unroll
    for (int i = 0; i < TILES; i++)
#pragma unroll
        for (int u = 0; u < 4; u++) *unit(tiles[i], row, 4 * half + u) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------- forward
template <int NB> struct FwdSmem {
    static constexpr int q = 0, k = q + NB * 16384, v = k + NB * 16384, h = v + 16384, y = h + NB * 8192,
                         x = y + 16384, total = x + (NB == 1 ? 16384 : 0);  // x: a part of w v that finds no room in q
};

template <typename T, int NB> __global__ void __launch_bounds__(256, 2) k_tc_fwd(const __grid_constant__ TcWalkArgs w) {
    extern __shared__ __align__(1024) char sm[];
    using L = FwdSmem<NB>;
    __shared__ Decays s_d;
    __shared__ __align__(8) uint64_t s_ld, s_m1, s_m2;
    __shared__ uint32_t s_tm, s_red[8];
    const Args& a = w.a;
    // thread: token (and accumulator row) tok, half `half` of its columns
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tok = tid & (C - 1), run = tok >> 5, half = tid >> 7;
    int64_t id = blockIdx.x;
    const int64_t ptiles = (a.P + PT - 1) / PT;
    const int64_t p0 = (id % ptiles) * PT;
    id /= ptiles;
    const int64_t h = id % a.H;
    id /= a.H;
    const int64_t seg = id % w.plan.K, b = id / w.plan.K;
    const int64_t hq = h / (a.H / a.G);
    const int64_t t_begin = seg * w.plan.seg, t_end = min(a.L, t_begin + w.plan.seg);
    const int64_t len = row_length(a, b);
    const int chunks = (int)((t_end - t_begin + C - 1) / C);
    char *Q = sm + L::q, *K = sm + L::k, *V = sm + L::v, *H = sm + L::h, *Y = sm + L::y;
    void* const W[3] = {Q, NB == 2 ? Q + 16384 : sm + L::x, Y};

    if (tid == 0) {
        mbar_init(&s_ld, 1);
        mbar_init(&s_m1, 1);
        mbar_init(&s_m2, 1);
        fence_proxy_async_smem();
    }
    if (warp == 0) tmem_alloc(&s_tm, 256);
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tm;
    // S, then (all of it read) P v and k^T (w v) in its place
    const uint32_t tS = tm, tOi = tm, tU = tm + 64, tP = tm + 128, tOe = tm + 192;
    const uint32_t my = (uint32_t)(run * 32) << 16;

    auto load = [&](int64_t t0) {
        mbar_expect_tx(&s_ld, (2 * NB + 1) * 16384);
#pragma unroll
        for (int n = 0; n < NB; n++) {
            tma_load_4d(K + n * 16384, &w.maps.k, n * 64, (int)hq, (int)t0, (int)b, &s_ld);
            tma_load_4d(Q + n * 16384, &w.maps.q, n * 64, (int)hq, (int)t0, (int)b, &s_ld);
        }
        tma_load_4d(V, &w.maps.v, (int)p0, (int)h, (int)t0, (int)b, &s_ld);
    };
    if (tid == 0) load(t_begin);

    float X[16 * NB];
    {
        const float* from = nullptr;
        if (w.plan.K > 1) from = w.seg_state + ((b * a.H + h) * w.plan.K + seg) * a.N * a.P;
        else if (w.init) from = w.init + (b * a.H + h) * a.N * a.P;
        load_state<NB>(from, a, p0, X);
    }
    auto valid = [&](int64_t t0) { return (int)max((int64_t)0, min((int64_t)C, len - t0)); };
    float g = load_g(a, b, h, t_begin, valid(t_begin));
    bool ok = true;
    int ch = 0;
    for (; ch < chunks; ch++) {
        const int64_t t0 = t_begin + (int64_t)ch * C;
        const int nv = valid(t0);
        float hs = 1.0f;  // scale of H as an operand
        if (kF16<T>) hs = f16_scale(block_max(state_max<NB>(X), s_red));
        put_state<T, NB>(H, nullptr, hs, X);
        const float rel = chunk_decays(s_d, g);
        if (ch + 1 < chunks) g = load_g(a, b, h, t0 + C, valid(t0 + C));
        ok = mbar_wait(&s_ld, ch & 1);
        if (ok && tok >= nv && t0 + tok < a.L) {
            if (NB == 2) {
                char* const t[5] = {Q, K, V, Q + 16384, K + 16384};
                clear_row<5>(t, tok, half);
            } else {
                char* const t[3] = {Q, K, V};
                clear_row<3>(t, tok, half);
            }
        }
        fence_proxy_async_smem();
        if (__syncthreads_or(!ok)) break;
        if (tid == 0) {
            tc_fence_after();
            constexpr uint32_t dS = mma_desc<T>(128, 128, false, false), dE = mma_desc<T>(128, PT, false, true);
#pragma unroll
            for (int s = 0; s < 4 * NB; s++) {
                const uint32_t at = (s >> 2) * 16384 + (s & 3) * 32;
                mma(tS, smem_desc(smem_addr(Q) + at), smem_desc(smem_addr(K) + at), dS, s > 0);
            }
#pragma unroll
            for (int s = 0; s < 4 * NB; s++) {
                const uint32_t at = (s >> 2) * 16384 + (s & 3) * 32;
                mma(tOe, smem_desc(smem_addr(Q) + at), smem_desc(smem_addr(H) + s * 2048), dE, s > 0);
            }
            bulk_wait_read();  // the last y has left its staging tile, which a part of w v takes below
            mma_commit(&s_m1);
        }
        float vs = 1.0f;
        if (kF16<T>) vs = f16_scale(block_max(row_max<T>(V, tok, half), s_red));
        Two end[4];
        run_ends(s_d, end);
        const Two mine = run == 0 ? end[0] : (run == 1 ? end[1] : (run == 2 ? end[2] : end[3]));
        const float ci = (mine.h - rel) + mine.l, cl = end[3].h + end[3].l;
        const float wt = ex2(two_diff(end[3], mine) + rel);
        ok = mbar_wait(&s_m1, ch & 1);
        tc_fence_after();
        // P, by runs of 32 columns, 16 to each half of the block: left of the diagonal e^{c_i - c_j} =
        // e^{c_i - c_e} e^{c_e - c_j} with e the end of the run (both factors are at most 1 for decays), on
        // it one exponential each
        float ps = 1.0f;
        if (kF16<T>) {
            float m = 0.0f;
            for (int cb = 0; cb <= run; cb++) {
                float s[32];
                tmem_ld32(tS + my + 32 * cb, s);
#pragma unroll
                for (int j = 0; j < 32; j++)
                    if (32 * cb + j <= tok) m = fmaxf(m, fabsf(s[j]));
            }
            ps = f16_scale(m);
        }
        for (int cb = 0; cb < 4; cb++) {
            uint32_t r[8];
            if (cb <= run) {
                float s[16];
                const int c0 = 32 * cb + 16 * half;
                tmem_ld16(tS + my + c0, s);
                if (cb < run) {
                    const Two e = cb == 0 ? end[0] : (cb == 1 ? end[1] : end[2]);
                    const float f = ps * ex2(two_diff(mine, e) - rel);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 t = *reinterpret_cast<const float4*>(&s_d.tail[c0 + j]);
                        r[j / 2] = pack2<T>(s[j] * (f * t.x), s[j + 1] * (f * t.y));
                        r[j / 2 + 1] = pack2<T>(s[j + 2] * (f * t.z), s[j + 3] * (f * t.w));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const int jj = 16 * half + j;
                        const float r0 = __shfl_sync(kFull, rel, jj), r1 = __shfl_sync(kFull, rel, jj + 1);
                        const float x = jj <= lane ? s[j] * (ps * ex2(r0 - rel)) : 0.0f;
                        const float y = jj + 1 <= lane ? s[j + 1] * (ps * ex2(r1 - rel)) : 0.0f;
                        r[j / 2] = pack2<T>(x, y);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++) r[j] = 0;
            }
            tmem_st8(tP + my + 16 * cb + 8 * half, r);
        }
        split_row<T>(V, tok, half, wt * vs, W[0], W[1], W[2]);
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        if (__syncthreads_or(!ok)) break;
        if (tid == 0) {
            tc_fence_after();
            constexpr uint32_t dV = mma_desc<T>(128, PT, false, true);
#pragma unroll
            for (int s = 0; s < C / 16; s++) mma_ts(tOi, tP + 8 * s, smem_desc(smem_addr(V) + s * 2048), dV, s > 0);
            const void* const parts[3] = {W[0], W[1], W[2]};
            mma_state<T, NB>(tU, K, parts);
            mma_commit(&s_m2);
        }
        ok = mbar_wait(&s_m2, ch & 1);
        tc_fence_after();
        if (tid == 0 && ok && ch + 1 < chunks) load(t0 + C);
        const float fe = a.scale * (ex2(ci) / hs), fi = a.scale / ps;
        {
            float e[32], o[32];
            tmem_ld32(tOe + my + 32 * half, e);
            tmem_ld32(tOi + my + 32 * half, o);
#pragma unroll
            for (int u = 0; u < 4; u++) {
                uint32_t r[4];
#pragma unroll
                for (int i = 0; i < 4; i++)
                    r[i] = pack2<T>(fmaf(fe, e[8 * u + 2 * i], fi * o[8 * u + 2 * i]),
                                    fmaf(fe, e[8 * u + 2 * i + 1], fi * o[8 * u + 2 * i + 1]));
                *unit(Y, tok, 4 * half + u) = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
        add_product<NB>(tU, ex2(cl), 1.0f / vs, X);
        tc_fence_before();
        fence_proxy_async_smem();
        if (__syncthreads_or(!ok)) break;
        if (tid == 0) {
            tma_store_4d(&w.maps.y, Y, (int)p0, (int)h, (int)t0, (int)b);
            bulk_commit();
        }
    }
    if (ch < chunks) {  // a wait ran out: report, wait for what is in flight (within limits), leave
        if (tid == 0) {
            atomicOr(w.status, kDevWaitTimeout);
            mbar_wait(&s_ld, ch & 1);
            mbar_wait(&s_ld, (ch + 1) & 1);
            mbar_wait(&s_m1, ch & 1);
            mbar_wait(&s_m2, ch & 1);
        }
    } else if (w.last && seg == w.plan.K - 1) {
        save_state<NB>(w.last + (b * a.H + h) * a.N * a.P, a, p0, X);
    }
    if (tid == 0) bulk_wait_all();
    __syncthreads();
    if (warp == 0) tmem_free(tm, 256);
}

// ---------------------------------------------------------------- states
// The walk without y: the end state of each segment (SUM), or the state before
// each chunk as operand tiles for the backward.
//   forward   X <- e^{cl} X + k^T (e^{cl - c} v)
//   reverse   X <- e^{cl} X + q^T (scale e^c dy), chunks last to first
template <int NB> struct StateSmem {
    static constexpr int k = 0, v = k + NB * 16384, w = v + 16384, total = w + 3 * 16384;
};

template <typename T, int NB, bool REV, bool SUM>
__global__ void __launch_bounds__(256, 2) k_tc_state(const __grid_constant__ TcWalkArgs w) {
    extern __shared__ __align__(1024) char sm[];
    using L = StateSmem<NB>;
    __shared__ Decays s_d;
    __shared__ __align__(8) uint64_t s_ld, s_m;
    __shared__ uint32_t s_tm, s_red[8];
    const Args& a = w.a;
    const int tid = threadIdx.x, warp = tid >> 5, tok = tid & (C - 1), run = tok >> 5, half = tid >> 7;
    int64_t id = blockIdx.x;
    const int64_t ptiles = (a.P + PT - 1) / PT;
    const int64_t pt = id % ptiles, p0 = pt * PT;
    id /= ptiles;
    const int64_t h = id % a.H;
    id /= a.H;
    const int64_t segs = SUM ? w.plan.K - 1 : w.plan.K;
    int64_t seg = id % segs;
    const int64_t b = id / segs;
    if (SUM && REV) seg += 1;
    const int64_t hq = h / (a.H / a.G);
    const int64_t t_begin = seg * w.plan.seg, t_end = min(a.L, t_begin + w.plan.seg);
    const int64_t len = row_length(a, b);
    const int chunks = (int)((t_end - t_begin + C - 1) / C);
    char *K = sm + L::k, *V = sm + L::v;
    void* const W[3] = {sm + L::w, sm + L::w + 16384, sm + L::w + 32768};

    if (tid == 0) {
        mbar_init(&s_ld, 1);
        mbar_init(&s_m, 1);
        fence_proxy_async_smem();
    }
    if (warp == 0) tmem_alloc(&s_tm, 64);
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tm;
    auto start_of = [&](int ch) { return t_begin + (int64_t)(REV ? chunks - 1 - ch : ch) * C; };
    auto valid = [&](int64_t t0) { return (int)max((int64_t)0, min((int64_t)C, len - t0)); };
    auto load = [&](int64_t t0) {
        mbar_expect_tx(&s_ld, (NB + 1) * 16384);
#pragma unroll
        for (int n = 0; n < NB; n++)
            tma_load_4d(K + n * 16384, REV ? &w.maps.q : &w.maps.k, n * 64, (int)hq, (int)t0, (int)b, &s_ld);
        tma_load_4d(V, REV ? &w.maps.dy : &w.maps.v, (int)p0, (int)h, (int)t0, (int)b, &s_ld);
    };
    if (tid == 0) load(start_of(0));
    float X[16 * NB];
    {
        const float* from = nullptr;
        if (!SUM && w.plan.K > 1) from = w.seg_state + ((b * a.H + h) * w.plan.K + seg) * a.N * a.P;
        else if (!SUM && w.init) from = w.init + (b * a.H + h) * a.N * a.P;
        load_state<NB>(from, a, p0, X);
    }
    float total = 0.0f, g = load_g(a, b, h, start_of(0), valid(start_of(0)));
    bool ok = true;
    int ch = 0;
    for (; ch < chunks; ch++) {
        const int64_t t0 = start_of(ch);
        const int nv = valid(t0);
        if (!SUM) {
            float s = 1.0f;
            if (kF16<T>) s = f16_scale(block_max(state_max<NB>(X), s_red));
            put_state<T, NB>(W[0], W[1], s, X);
            fence_proxy_async_smem();
            __syncthreads();
            if (tid == 0) {
                const int64_t at = ((b * a.H + h) * ptiles + pt) * w.chunks + t0 / C;
                char* to = static_cast<char*>(w.images) + at * (2 * NB * 8192);
                bulk_store(to, W[0], NB * 8192);
                bulk_store(to + NB * 8192, W[1], NB * 8192);
                bulk_commit();
                if (kF16<T>) w.image_scale[at] = s;
                bulk_wait_read();
            }
        }
        const float rel = chunk_decays(s_d, g);
        if (ch + 1 < chunks) g = load_g(a, b, h, start_of(ch + 1), valid(start_of(ch + 1)));
        ok = mbar_wait(&s_ld, ch & 1);
        if (ok && tok >= nv && t0 + tok < a.L) {
            if (NB == 2) {
                char* const t[3] = {K, V, K + 16384};
                clear_row<3>(t, tok, half);
            } else {
                char* const t[2] = {K, V};
                clear_row<2>(t, tok, half);
            }
            fence_proxy_async_smem();
        }
        if (__syncthreads_or(!ok)) break;
        float vs = 1.0f;
        if (kF16<T>) vs = f16_scale(block_max(row_max<T>(V, tok, half), s_red));
        Two end[4];
        run_ends(s_d, end);
        const Two mine = run == 0 ? end[0] : (run == 1 ? end[1] : (run == 2 ? end[2] : end[3]));
        const float cl = end[3].h + end[3].l;
        split_row<T>(V, tok, half, vs * ex2(REV ? (mine.h - rel) + mine.l : two_diff(end[3], mine) + rel), W[0], W[1], W[2]);
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            const void* const parts[3] = {W[0], W[1], W[2]};
            mma_state<T, NB>(tm, K, parts);
            mma_commit(&s_m);
        }
        ok = mbar_wait(&s_m, ch & 1);
        tc_fence_after();
        if (tid == 0 && ok && ch + 1 < chunks) load(start_of(ch + 1));
        add_product<NB>(tm, ex2(cl), (REV ? a.scale : 1.0f) / vs, X);
        total += cl;
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;
    }
    if (ch < chunks) {
        if (tid == 0) {
            atomicOr(w.status, kDevWaitTimeout);
            mbar_wait(&s_ld, ch & 1);
            mbar_wait(&s_ld, (ch + 1) & 1);
            mbar_wait(&s_m, ch & 1);
        }
    } else if (SUM) {
        save_state<NB>(w.seg_state + ((b * a.H + h) * w.plan.K + seg) * a.N * a.P, a, p0, X);
        if (tid == 0 && pt == 0) w.seg_decay[(b * a.H + h) * w.plan.K + seg] = total / kLog2e;
    } else if (w.last && seg == (REV ? 0 : w.plan.K - 1)) {
        save_state<NB>(w.last + (b * a.H + h) * a.N * a.P, a, p0, X);
    }
    if (tid == 0) bulk_wait_all();
    __syncthreads();
    if (warp == 0) tmem_free(tm, 64);
}

unsigned blocks(const TcWalkArgs& w, int64_t segs) {
    return (unsigned)(ceil_div(w.a.P, PT) * w.a.H * w.a.Bsz * segs);
}

template <typename K> cudaError_t go(K kernel, int smem, unsigned grid, const TcWalkArgs& w, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, 256, smem, st>>>(w);
    return cudaGetLastError();
}

template <typename T, int NB> cudaError_t fwd_n(const TcWalkArgs& w, cudaStream_t st) {
    return go(k_tc_fwd<T, NB>, FwdSmem<NB>::total, blocks(w, w.plan.K), w, st);
}
template <typename T, int NB> cudaError_t state_n(const TcWalkArgs& w, bool reverse, bool sum, cudaStream_t st) {
    const unsigned grid = blocks(w, sum ? w.plan.K - 1 : w.plan.K);
    constexpr int smem = StateSmem<NB>::total;
    if (reverse) return sum ? go(k_tc_state<T, NB, true, true>, smem, grid, w, st) : go(k_tc_state<T, NB, true, false>, smem, grid, w, st);
    return sum ? go(k_tc_state<T, NB, false, true>, smem, grid, w, st) : go(k_tc_state<T, NB, false, false>, smem, grid, w, st);
}

}  // namespace

cudaError_t launch_tc_fwd(const TcWalkArgs& w, cudaStream_t st) {
    const bool wide = w.a.N > 64;
    if (w.a.dtype == 1) return wide ? fwd_n<__half, 2>(w, st) : fwd_n<__half, 1>(w, st);
    return wide ? fwd_n<__nv_bfloat16, 2>(w, st) : fwd_n<__nv_bfloat16, 1>(w, st);
}

cudaError_t launch_tc_state(const TcWalkArgs& w, bool reverse, bool sum, cudaStream_t st) {
    const bool wide = w.a.N > 64;
    if (w.a.dtype == 1) return wide ? state_n<__half, 2>(w, reverse, sum, st) : state_n<__half, 1>(w, reverse, sum, st);
    return wide ? state_n<__nv_bfloat16, 2>(w, reverse, sum, st) : state_n<__nv_bfloat16, 1>(w, reverse, sum, st);
}

}  // namespace la
}  // namespace ss
