// Linear attention on the tensor cores: the forward, and the states at the
// chunks' borders that the backward reads.  16-bit io.
//
// A chunk is 128 tokens (the M of a matrix product).  With c_i the cumulative
// log decay inside the chunk, cl its end and H the state before it:
//   S = q k^T,  P_ij = e^{c_i - c_j} S_ij (j <= i),  y = scale (e^{c_i} q H + P v)
//   H <- e^{cl} H + k^T (e^{cl - c} v)
// One block walks one segment of one (batch row, head, 64 value channels): S,
// q H and k^T (w v) are products of tiles that TMA brought, P is the left
// operand out of tensor memory.  Two warpgroups share a chunk after S and q H:
// the state half makes w v, adds k^T (w v) to H, which it keeps in f32 registers
// (thread = one of the N rows), and writes the next chunk's H operand; the
// output half makes P, P v and y.  Their chains overlap (a chunk took 10.5 thousand
// cycles when all threads did all of it in turn, 4.8 so).
//
// Roundings to 16 bits: P, and H as an operand of q H (one rounding of terms of a
// 16-bit y each).  The state is f32: w v enters as two or three 16-bit parts whose
// sum holds 22 to 24 bits.
//
// Measured, bf16.  4 x 4096 tokens, 80 heads, N 128, P 64: sums 17 us, carries 9,
// forward 186 (DRAM 22 %, tensor cores 35 %, issue 43 %, shared memory of the threads
// alone 35 %): bound by the chain of a chunk, of which the two blocks an SM has room
// for (at N = 128 by shared memory) hide half.  131072 tokens, 16 heads, N 64: sums
// 112 us and forward 234, both at 57 % of DRAM's rate; the sums read k and v once
// more, which is what one sequence's parallelism costs.  f16's scales take 3 to 4 %
// more (8 x 2047 ragged tokens, 20 heads: 112 us, 108 with scales of the undecayed
// values, which leave f16's range when g is positive).
#include "la_tc.h"
#include "../simd.cuh"
#include "tc.cuh"

namespace ss {
namespace la {
namespace {

constexpr int C = kChunkTc;
constexpr int PT = kTileP;

// 16-bit parts of w v: 3 x 8 bits (bf16), 2 x 11 (f16)
template <typename T> constexpr int kParts = kF16<T> ? 2 : 3;

// The chunk's decays, by runs of 32 tokens (one warp's): c_i = (the run's end) -
// rel_i with rel a thread's own.  Shared: tail = e^{rel}, its largest value in each
// run (each where wanted) and the log2 decay of each run.
// A warpgroup (token = tid % 128), g: the token's log decay.  Returns rel (at
// most 0 for decays).
__device__ __forceinline__ float chunk_decays(float* tail, float* top, Two* total, float g) {
    const int tok = threadIdx.x & (C - 1);
    const float in[1] = {clamp_g(g) * kLog2e};
    Two c[1];
    warp_cumsum<1>(in, c);
    const Two end = {__shfl_sync(kFull, c[0].h, 31), __shfl_sync(kFull, c[0].l, 31)};
    const float rel = two_diff(end, c[0]);
    if (tail) {
        const float t = ex2(rel);
        tail[tok] = t;
        if (top) {
            uint32_t m;
            asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(__float_as_uint(t)));
            if ((tok & 31) == 0) top[tok >> 5] = __uint_as_float(m);
        }
    }
    if ((tok & 31) == 31) total[tok >> 5] = end;
    return rel;
}
// After a barrier: log2 decays from the chunk's start to the end of each run.
__device__ __forceinline__ void run_ends(const Two* total, Two (&end)[4]) {
    end[0] = total[0];
#pragma unroll
    for (int i = 1; i < 4; i++) end[i] = two_add(end[i - 1], total[i]);
}
// The token's log decay as it is in memory: nothing waits for it until it is used.
__device__ __forceinline__ float load_g(const Args& a, int64_t b, int64_t h, int64_t t0, int nv) {
    const int t = threadIdx.x & (C - 1);
    return t < nv ? a.g[a.g_per_head ? h : (b * a.L + t0 + t) * a.H + h] : 0.0f;
}

// Barrier of one warpgroup (128 threads): id 1 or 2.
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// Largest value of a warpgroup's threads (all get it); v >= 0.  Two barriers.
__device__ __forceinline__ float group_max(float v, uint32_t* red, int id) {
    uint32_t m;
    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(__float_as_uint(v)));
    if ((threadIdx.x & 31) == 0) red[(threadIdx.x >> 5) & 3] = m;
    group_sync(id);
    m = max(max(red[0], red[1]), max(red[2], red[3]));
    group_sync(id);
    return __uint_as_float(m);
}

// (x, y) as a pair of 16-bit values, and what the pair leaves of them.  bf16
// truncates (the rest is exact, and keeps the sign), so that three parts hold
// all 24 bits; f16 rounds, two parts hold 22.
template <typename T> __device__ __forceinline__ uint32_t split2(float2& f) {
    if (kF16<T>) {
        const uint32_t r = pack2<T>(f.x, f.y);
        f = fma2(unpack2<T>(r), splat2(-1.0f), f);
        return r;
    }
    const uint32_t x = __float_as_uint(f.x), y = __float_as_uint(f.y);
    f = fma2(make_float2(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u)), splat2(-1.0f), f);
    return __byte_perm(x, y, 0x7632);
}

// 16-byte units u0 .. u1 - 1 of row `row` of a value tile, times w, as 16-bit
// parts (same layout).
template <typename T>
__device__ __forceinline__ void split_row(void* v, int row, int u0, int u1, float w, void* p0, void* p1, void* p2) {
#pragma unroll 2
    for (int u = u0; u < u1; u++) {
        const uint4 in = *unit(v, row, u);
        const uint32_t x[4] = {in.x, in.y, in.z, in.w};
        uint32_t r[3][4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float2 f = mul2(unpack2<T>(x[i]), splat2(w));
            r[0][i] = split2<T>(f);
            if (kParts<T> == 3) {
                r[1][i] = split2<T>(f);
                r[2][i] = pack2<T>(f.x, f.y);
            } else {
                r[1][i] = pack2<T>(f.x, f.y);
            }
        }
        *unit(p0, row, u) = make_uint4(r[0][0], r[0][1], r[0][2], r[0][3]);
        *unit(p1, row, u) = make_uint4(r[1][0], r[1][1], r[1][2], r[1][3]);
        if (kParts<T> == 3) *unit(p2, row, u) = make_uint4(r[2][0], r[2][1], r[2][2], r[2][3]);
    }
}

template <typename T> __device__ __forceinline__ float row_max(void* v, int row, int half) {  // units 4 half .. + 3
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

// The part of the state that one of TH threads (128 or 256, aligned in the block)
// holds: a row, W adjacent columns.  NB == 1: the product's 128 rows hold the 64
// twice, so that a thread's row is in its own lane.
template <int NB, int TH> struct StateOf {
    static constexpr int W = 64 * 64 * NB / TH;
    __device__ static int row() { return threadIdx.x & (64 * NB - 1); }
    __device__ static int col() { return (int)(threadIdx.x & (TH - 1)) / (64 * NB) * W; }
};

__device__ __forceinline__ void tmem_ldw(uint32_t addr, float (&x)[16]) { tmem_ld16(addr, x); }
__device__ __forceinline__ void tmem_ldw(uint32_t addr, float (&x)[32]) { tmem_ld32(addr, x); }

// A state tile in memory: rows of `stride` floats, `cols` of the 64 columns exist.
struct StateTile {
    const float* p;  // null: zero
    int64_t rows, stride, cols;
};
template <int NB, int TH> __device__ __forceinline__ void load_state(const StateTile& s, float (&X)[StateOf<NB, TH>::W]) {
    const int n = StateOf<NB, TH>::row(), c0 = StateOf<NB, TH>::col();
#pragma unroll
    for (int c = 0; c < StateOf<NB, TH>::W; c += 4) {
        float4 f = {0.0f, 0.0f, 0.0f, 0.0f};
        if (s.p && n < s.rows && c0 + c < s.cols) f = *reinterpret_cast<const float4*>(s.p + n * s.stride + c0 + c);
        X[c] = f.x;
        X[c + 1] = f.y;
        X[c + 2] = f.z;
        X[c + 3] = f.w;
    }
}
template <int NB, int TH> __device__ __forceinline__ void save_state(const StateTile& s, const float (&X)[StateOf<NB, TH>::W]) {
    const int n = StateOf<NB, TH>::row(), c0 = StateOf<NB, TH>::col();
#pragma unroll
    for (int c = 0; c < StateOf<NB, TH>::W; c += 4)
        if (n < s.rows && c0 + c < s.cols)
            *reinterpret_cast<float4*>(const_cast<float*>(s.p) + n * s.stride + c0 + c) =
                make_float4(X[c], X[c + 1], X[c + 2], X[c + 3]);
}

// A unit's place, and the walk a block takes, from its index.
struct Walk {
    int64_t b, h, hq, pt, p0, cut, seg, t_begin, t_end;
    bool is_cut, reverse;

    __device__ void place(const TcWalkArgs& w, int64_t unit) {
        const Args& a = w.a;
        const int64_t ptiles = (a.P + PT - 1) / PT, units = a.Bsz * a.H * ptiles;
        reverse = unit >= units;
        if (reverse) unit -= units;
        pt = unit % ptiles;
        p0 = pt * PT;
        h = unit / ptiles % a.H;
        b = unit / ptiles / a.H;
        hq = h / (a.H / a.G);
    }
    __device__ Walk() {}
    __device__ Walk(const TcWalkArgs& w, bool sum) {
        int64_t id = blockIdx.x, unit = id;
        is_cut = sum || id >= w.plan.whole;
        cut = seg = 0;
        if (is_cut) {
            if (!sum) id -= w.plan.whole;
            cut = id % w.plan.cut;
            seg = id / w.plan.cut;
            unit = w.plan.whole + cut;
        }
        place(w, unit);
        if (sum && reverse) seg += 1;  // the segment walked last needs no sum
        t_begin = is_cut ? seg * w.plan.seg : 0;
        t_end = is_cut ? min(w.a.L, t_begin + w.plan.seg) : w.a.L;
    }
    __device__ const TcDir& dir(const TcWalkArgs& w) const { return w.dir[reverse]; }
    __device__ StateTile start(const TcWalkArgs& w) const { return is_cut ? segment(w) : whole(w, dir(w).init); }
    __device__ StateTile segment(const TcWalkArgs& w) const {
        return {w.seg_state + (cut * w.plan.K + seg) * w.a.N * PT, w.a.N, PT, PT};
    }
    __device__ StateTile whole(const TcWalkArgs& w, const float* p) const {
        return {p ? p + (b * w.a.H + h) * w.a.N * w.a.P + p0 : nullptr, w.a.N, w.a.P, w.a.P - p0};
    }
    // where its last state goes, if that is the whole walk's
    __device__ float* last(const TcWalkArgs& w) const {
        return !is_cut || seg == (reverse ? 0 : w.plan.K - 1) ? dir(w).last : nullptr;
    }
};
template <int W> __device__ __forceinline__ float state_max(const float (&X)[W]) {
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < W; c++) m = fmaxf(m, fabsf(X[c]));
    return m;
}
// X <- d X + u * (the sum of PARTS products, 64 columns apart in tensor memory)
template <int NB, int TH, int PARTS>
__device__ __forceinline__ void add_product(uint32_t tm, float d, float u, float (&X)[StateOf<NB, TH>::W]) {
    constexpr int W = StateOf<NB, TH>::W, B = W < 32 ? W : 32;
#pragma unroll
    for (int c = 0; c < W; c += B) {
#pragma unroll
        for (int p = 0; p < PARTS; p++) {
            float f[B];
            tmem_ldw(tm + ((threadIdx.x & 96) << 16) + StateOf<NB, TH>::col() + c + 64 * p, f);
#pragma unroll
            for (int i = 0; i < B; i += 2) {
                float2 y = make_float2(X[c + i], X[c + i + 1]);
                if (p == 0) y = mul2(splat2(d), y);
                y = fma2(splat2(u), make_float2(f[i], f[i + 1]), y);
                X[c + i] = y.x;
                X[c + i + 1] = y.y;
            }
        }
    }
}
// 16-bit rows [n][p] of X * s: an operand tile, and PARTS - 1 more, one after the
// other, of what the rounding left
template <typename T, int NB, int TH, int PARTS>
__device__ __forceinline__ void put_state(char* to, float s, const float (&X)[StateOf<NB, TH>::W]) {
    const int n = StateOf<NB, TH>::row(), u0 = StateOf<NB, TH>::col() / 8;
#pragma unroll
    for (int u = 0; u < StateOf<NB, TH>::W / 8; u++) {
        uint32_t r[PARTS][4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float2 f = make_float2(X[8 * u + 2 * i], X[8 * u + 2 * i + 1]);
            if (kF16<T>) f = mul2(f, splat2(s));
#pragma unroll
            for (int p = 0; p < PARTS; p++) {
                r[p][i] = pack2<T>(f.x, f.y);
                if (p + 1 < PARTS) f = fma2(unpack2<T>(r[p][i]), splat2(-1.0f), f);
            }
        }
#pragma unroll
        for (int p = 0; p < PARTS; p++) *unit(to + p * NB * 8192, n, u0 + u) = make_uint4(r[p][0], r[p][1], r[p][2], r[p][3]);
    }
}

// k^T (w v): rows n (both halves of the 128 rows the same 64 when NB == 1), columns
// p.  Its parts added up in 64 columns of tensor memory (w: one tile per part), the
// smallest first: each step's rounding goes with what has been added so far, and the
// last state is off by 1.5e-7 instead of 1.4e-6 (bf16, 1000 tokens) ...
template <typename T, int NB> __device__ __forceinline__ void mma_state(uint32_t tm, const void* k, const void* const (&w)[3]) {
    constexpr uint32_t desc = mma_desc<T>(128, PT, true, true);
    const uint32_t ka = smem_addr(k);
#pragma unroll
    for (int p = kParts<T> - 1; p >= 0; p--)
#pragma unroll
        for (int s = 0; s < C / 16; s++)
            mma(tm, smem_desc(ka + s * 2048, NB == 2 ? 16384 : 0), smem_desc(smem_addr(w[p]) + s * 2048), desc, p < kParts<T> - 1 || s > 0);
}
// ... or side by side (w: the parts' tiles one after the other), which reads k once
template <typename T, int NB> __device__ __forceinline__ void mma_state_wide(uint32_t tm, const void* k, const void* w) {
    constexpr uint32_t desc = mma_desc<T>(128, PT * kParts<T>, true, true);
    const uint32_t ka = smem_addr(k), wa = smem_addr(w);
#pragma unroll
    for (int s = 0; s < C / 16; s++)
        mma(tm, smem_desc(ka + s * 2048, NB == 2 ? 16384 : 0), smem_desc(wa + s * 2048, 16384), desc, s > 0);
}

// A row of each tile that a copy filled with a token beyond the batch row's length: zero.
template <int TILES> __device__ __forceinline__ void clear_row(char* const (&tiles)[TILES], int row) {
#pragma unroll
    for (int i = 0; i < TILES; i++)
#pragma unroll
        for (int u = 0; u < 8; u++) *unit(tiles[i], row, u) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------- forward
template <int NB> struct FwdSmem {
    static constexpr int q = 0, k = q + NB * 16384, v = k + NB * 16384, h = v + 16384, y = h + NB * 8192,
                         x = y + 16384, total = x + (NB == 1 ? 16384 : 0);  // x: a part of w v that finds no room in q
};

template <typename T, int NB> __global__ void __launch_bounds__(256, 2) k_tc_fwd(const __grid_constant__ TcWalkArgs w) {
    extern __shared__ __align__(1024) char sm[];
    using L = FwdSmem<NB>;
    __shared__ float s_tail[C], s_top[4];
    __shared__ Two s_total[2][4];
    // copies landed; S; q H; P v; k^T (w v)
    __shared__ __align__(8) uint64_t s_ld, s_mS, s_mE, s_mO, s_mU;
    __shared__ uint32_t s_tm, s_red[4], s_fail;
    __shared__ float s_hs[2];
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, tok = tid & (C - 1), run = tok >> 5;
    const bool out = tid >= C;  // output half, else state half
    const Walk at(w, false);
    const int64_t b = at.b, h = at.h, hq = at.hq, p0 = at.p0, t_begin = at.t_begin, t_end = at.t_end;
    const int64_t len = row_length(a, b);
    const int chunks = (int)((t_end - t_begin + C - 1) / C);
    char *Q = sm + L::q, *K = sm + L::k, *V = sm + L::v, *H = sm + L::h, *Y = sm + L::y;
    void* const W[3] = {Q, NB == 2 ? Q + 16384 : sm + L::x, Y};

    if (tid == 0) {
        mbar_init(&s_ld, 1);
        mbar_init(&s_mS, 1);
        mbar_init(&s_mE, 1);
        mbar_init(&s_mO, 1);
        mbar_init(&s_mU, 1);
        s_fail = 0;
        fence_proxy_async_smem();
    }
    if (tid < 32) tmem_alloc(&s_tm, 256);
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tm;
    // S; P in the place of its first 64 columns, P v in the others'
    const uint32_t tS = tm, tP = tm, tO = tm + 64, tE = tm + 128, tU = tm + 192;
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
    auto prefetch = [&](int64_t t0) {
#pragma unroll
        for (int n = 0; n < NB; n++) {
            tma_prefetch_4d(&w.maps.k, n * 64, (int)hq, (int)t0, (int)b);
            tma_prefetch_4d(&w.maps.q, n * 64, (int)hq, (int)t0, (int)b);
        }
        tma_prefetch_4d(&w.maps.v, (int)p0, (int)h, (int)t0, (int)b);
    };
    auto valid = [&](int64_t t0) { return (int)max((int64_t)0, min((int64_t)C, len - t0)); };
    if (tid == C) load(t_begin);

    float g = load_g(a, b, h, t_begin, valid(t_begin));
    bool ok = true;
    int ch = 0;
    // both halves: chunk ch's decays (into end, rel), then its tiles
    auto decays = [&](float* tail, Two* total, int64_t t0) {
        const float rel = chunk_decays(tail, kF16<T> ? s_top : nullptr, total, g);
        if (ch + 1 < chunks) g = load_g(a, b, h, t0 + C, valid(t0 + C));
        return rel;
    };
    auto end_of = [&](const Two (&end)[4]) { return run == 0 ? end[0] : (run == 1 ? end[1] : (run == 2 ? end[2] : end[3])); };
    if (!out) {
        float X[StateOf<NB, 128>::W];
        load_state<NB, 128>(at.start(w), X);
        for (; ch < chunks; ch++) {
            const uint32_t ph = ch & 1;
            float hs = 1.0f;  // scale of H as an operand
            if (kF16<T>) {
                hs = f16_scale(group_max(state_max(X), s_red, 1));
                if (tid == 0) s_hs[ph] = hs;
            }
            put_state<T, NB, 128, 1>(H, hs, X);
            const float rel = decays(nullptr, s_total[0], t_begin + (int64_t)ch * C);
            ok = ok && mbar_wait(&s_ld, ph);
            fence_proxy_async_smem();
            if (__syncthreads_or(!ok)) break;
            Two end[4];
            run_ends(s_total[0], end);
            const Two mine = end_of(end);
            const float wt = ex2(two_diff(end[3], mine) + rel), cl = end[3].h + end[3].l;
            if (tid == 0) {  // (this half waits for both; the other's P must not)
                tc_fence_after();
                constexpr uint32_t dS = mma_desc<T>(128, 128, false, false), dE = mma_desc<T>(128, PT, false, true);
#pragma unroll
                for (int s = 0; s < 4 * NB; s++) {
                    const uint32_t at = (s >> 2) * 16384 + (s & 3) * 32;
                    mma(tS, smem_desc(smem_addr(Q) + at), smem_desc(smem_addr(K) + at), dS, s > 0);
                }
                mma_commit(&s_mS);
#pragma unroll
                for (int s = 0; s < 4 * NB; s++) {
                    const uint32_t at = (s >> 2) * 16384 + (s & 3) * 32;
                    mma(tE, smem_desc(smem_addr(Q) + at), smem_desc(smem_addr(H) + s * 2048), dE, s > 0);
                }
                mma_commit(&s_mE);
            }
            __syncwarp();
            float vs = 1.0f;
            if (kF16<T>) vs = f16_scale(group_max(wt * fmaxf(row_max<T>(V, tok, 0), row_max<T>(V, tok, 1)), s_red, 1));
            ok = mbar_wait(&s_mE, ph);  // q makes room for w v
            split_row<T>(V, tok, 0, 8, wt * vs, W[0], W[1], W[2]);
            fence_proxy_async_smem();
            group_sync(1);
            if (tid == 0) {
                tc_fence_after();
                const void* const parts[3] = {W[0], W[1], W[2]};
                mma_state<T, NB>(tU, K, parts);
                mma_commit(&s_mU);
            }
            ok = mbar_wait(&s_mU, ph) && ok;
            tc_fence_after();
            add_product<NB, 128, 1>(tU, ex2(cl), 1.0f / vs, X);
            tc_fence_before();
        }
        if (ch == chunks && at.last(w)) save_state<NB, 128>(at.whole(w, at.last(w)), X);
    } else {
        for (; ch < chunks; ch++) {
            const int64_t t0 = t_begin + (int64_t)ch * C;
            const uint32_t ph = ch & 1;
            const float rel = decays(s_tail, s_total[1], t0);
            ok = ok && mbar_wait(&s_ld, ph);
            if (ok && tok >= valid(t0) && t0 + tok < a.L) {
                if (NB == 2) {
                    char* const t[5] = {Q, K, V, Q + 16384, K + 16384};
                    clear_row<5>(t, tok);
                } else {
                    char* const t[3] = {Q, K, V};
                    clear_row<3>(t, tok);
                }
            }
            fence_proxy_async_smem();
            if (tid == C) {
                bulk_wait_read();  // the last y has left its staging tile, which a part of w v takes
                if (ch + 1 < chunks) prefetch(t0 + C);
            }
            if (__syncthreads_or(!ok)) break;
            Two end[4];
            run_ends(s_total[1], end);
            const Two mine = end_of(end);
            const float ci = (mine.h - rel) + mine.l;
            float lift = 1.0f;  // largest e^{c_i - c_j} of the token's row (1 for decays)
            if (kF16<T>) {
                float top = rel;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float x = __shfl_up_sync(kFull, top, o);
                    if (lane >= o) top = fmaxf(top, x);
                }
                lift = ex2(top - rel);
#pragma unroll
                for (int cb = 0; cb < 3; cb++)
                    if (cb < run) lift = fmaxf(lift, ex2(two_diff(mine, end[cb]) - rel) * s_top[cb]);
            }
            ok = mbar_wait(&s_mS, ph);
            tc_fence_after();
            // P, by runs of 32 columns: left of the diagonal e^{c_i - c_j} = e^{c_i - c_e} e^{c_e - c_j} with e
            // the end of the run (both factors are at most 1 for decays), on it one exponential each
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
                ps = f16_scale(m * lift);
            }
            for (int cb = 0; cb < 4; cb++) {
                uint32_t r[16];
                if (cb <= run) {
                    float s[32];
                    tmem_ld32(tS + my + 32 * cb, s);
                    if (cb < run) {
                        const Two e = cb == 0 ? end[0] : (cb == 1 ? end[1] : end[2]);
                        const float2 f = splat2(ps * ex2(two_diff(mine, e) - rel));
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 t = *reinterpret_cast<const float4*>(&s_tail[32 * cb + j]);
                            const float2 x = mul2(make_float2(s[j], s[j + 1]), mul2(f, make_float2(t.x, t.y)));
                            const float2 y = mul2(make_float2(s[j + 2], s[j + 3]), mul2(f, make_float2(t.z, t.w)));
                            r[j / 2] = pack2<T>(x.x, x.y);
                            r[j / 2 + 1] = pack2<T>(y.x, y.y);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float r0 = __shfl_sync(kFull, rel, j), r1 = __shfl_sync(kFull, rel, j + 1);
                            const float x = j <= lane ? s[j] * (ps * ex2(r0 - rel)) : 0.0f;
                            const float y = j + 1 <= lane ? s[j + 1] * (ps * ex2(r1 - rel)) : 0.0f;
                            r[j / 2] = pack2<T>(x, y);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j++) r[j] = 0;
                }
                tmem_st16(tP + my + 16 * cb, r);
            }
            tmem_wait_st();
            tc_fence_before();
            group_sync(2);
            if (tid == C) {
                tc_fence_after();
                constexpr uint32_t dV = mma_desc<T>(128, PT, false, true);
#pragma unroll
                for (int s = 0; s < C / 16; s++) mma_ts(tO, tP + 8 * s, smem_desc(smem_addr(V) + s * 2048), dV, s > 0);
                mma_commit(&s_mO);
            }
            ok = mbar_wait(&s_mE, ph) && ok;
            tc_fence_after();
            // past the row's length: zero rows times a state or a v that is not finite are not zero
            const bool counts = tok < valid(t0);
            const float fe = a.scale * (kF16<T> ? ex2(ci) / s_hs[ph] : ex2(ci)), fi = kF16<T> ? a.scale / ps : a.scale;
            ok = mbar_wait(&s_mO, ph) && ok;
            ok = mbar_wait(&s_mU, ph) && ok;  // w v has left the staging tile, k and v are done with
            tc_fence_after();
            if (tid == C && ok && ch + 1 < chunks) load(t0 + C);
#pragma unroll
            for (int half = 0; half < 2; half++) {
                float e[32], o[32];
                tmem_ld32(tE + my + 32 * half, e);
                tmem_ld32(tO + my + 32 * half, o);
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    uint32_t r[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int c = 8 * u + 2 * i;
                        const float2 x = fma2(splat2(fi), make_float2(o[c], o[c + 1]),
                                              mul2(splat2(fe), make_float2(e[c], e[c + 1])));
                        r[i] = counts ? pack2<T>(x.x, x.y) : 0;
                    }
                    *unit(Y, tok, 4 * half + u) = make_uint4(r[0], r[1], r[2], r[3]);
                }
            }
            tc_fence_before();
            fence_proxy_async_smem();
            group_sync(2);
            if (tid == C) {
                tma_store_4d(&w.maps.y, Y, (int)p0, (int)h, (int)t0, (int)b);
                bulk_commit();
            }
        }
    }
    if (!ok) s_fail = 1;  // a wait ran out, in the last chunk or (everybody left the loop then) before
    if (tid == C) bulk_wait_all();
    uint64_t* const bars[] = {&s_ld, &s_mS, &s_mE, &s_mO, &s_mU};
    end_block(&s_fail, w.status, bars, tm, 256);
}

// ---------------------------------------------------------------- states
// The walk without y: the end state of each segment (SUM), or the state before
// each chunk as operand tiles for the backward.
//   forward   X <- e^{cl} X + k^T (e^{cl - c} v)
//   reverse   X <- e^{cl} X + q^T (scale e^c dy), chunks last to first
//
// Two chunks are in work at a time (and the copies of the next under way), each
// part of the block on its own: 8 warps make w v, 8 keep the state (add a chunk's
// product to it, write it out as an image), one makes the weights w, one issues copies
// and products.
// Measured, bf16, 2 x 4096 tokens, 80 heads, N 128, P 64, both directions: 115 us (183 MB
// read, 278 written and 84 more kept in the L2 cache: half of DRAM's rate; 117 us without
// the prefetch, 132 with the image stored from registers); a chunk takes 3200 cycles, of
// which the shared memory's traffic (256 KB) alone 2000, and no part of its chain left
// out takes more than 15 us off.
template <int NB, int PARTS> struct StateSmem {
    static constexpr int ring = NB == 1 ? 3 : 2;  // chunks whose k and v are here or on their way
    static constexpr int k = 0, v = k + NB * 16384, stage = v + 16384, w = ring * stage, parts = 3 * 16384,
                         image = w + 2 * parts, total = image + PARTS * NB * 8192;
};
constexpr int kSplit = 256, kKeep = 256, kStateThreads = kSplit + kKeep + 64;

template <typename T, int NB, bool SUM>
__global__ void __launch_bounds__(kStateThreads, 1) k_tc_state(const __grid_constant__ TcWalkArgs w) {
    extern __shared__ __align__(1024) char sm[];
    constexpr int kImage = kImageParts<kF16<T>, NB>;
    using L = StateSmem<NB, kImage>;
    __shared__ float s_weight[2][C], s_all[2], s_vs[2];  // w and e^{cl} of a stage's chunk
    // copies landed (of a ring's place); w made; w v made; product done; product read (of a stage)
    __shared__ __align__(8) uint64_t s_ld[L::ring], s_g[2], s_w[2], s_u[2], s_free[2];
    __shared__ uint32_t s_tm, s_red[2][4], s_most[8], s_fail;
    const Args& a = w.a;
    const int tid = threadIdx.x;
    const Walk at(w, SUM);
    const bool REV = at.reverse;
    const int64_t b = at.b, h = at.h, t_begin = at.t_begin, t_end = at.t_end;
    const int64_t len = row_length(a, b);
    const int chunks = (int)((t_end - t_begin + C - 1) / C);

    if (tid == 0) {
#pragma unroll
        for (int s = 0; s < L::ring; s++) mbar_init(&s_ld[s], 1);
#pragma unroll
        for (int s = 0; s < 2; s++) {
            mbar_init(&s_g[s], 32);
            mbar_init(&s_w[s], kSplit);
            mbar_init(&s_u[s], 1);
            mbar_init(&s_free[s], kKeep);
        }
        s_fail = 0;
        fence_proxy_async_smem();
    }
    if (tid < 32) tmem_alloc(&s_tm, 512);
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tm;
    auto start_of = [&](int ch) { return t_begin + (int64_t)(REV ? chunks - 1 - ch : ch) * C; };
    auto valid = [&](int64_t t0) { return (int)max((int64_t)0, min((int64_t)C, len - t0)); };

    if (tid < kSplit) {  // ---------------- w v, half a row (four 16-byte units) a thread
        const int tok = tid & (C - 1), half = tid >> 7;
        for (int ch = 0; ch < chunks; ch++) {
            const int s = ch & 1;
            const uint32_t ph = (ch >> 1) & 1;
            const int64_t t0 = start_of(ch);
            char *K = sm + (ch % L::ring) * L::stage + L::k, *V = sm + (ch % L::ring) * L::stage + L::v;
            char* W = sm + L::w + s * L::parts;
            wait_or_fail(&s_g[s], ph, &s_fail);  // (made after the stage's last product was read)
            wait_or_fail(&s_ld[ch % L::ring], (ch / L::ring) & 1, &s_fail);
            if (tok >= valid(t0) && t0 + tok < a.L) {
#pragma unroll
                for (int u = 4 * half; u < 4 * half + 4; u++) {
#pragma unroll
                    for (int n = 0; n < NB; n++) *unit(K + n * 16384, tok, u) = make_uint4(0, 0, 0, 0);
                    *unit(V, tok, u) = make_uint4(0, 0, 0, 0);
                }
            }
            float wt = s_weight[s][tok];
            if (kF16<T>) {
                // one scale for the tile: the larger of both halves' largest w v
                const float m = group_max(wt * row_max<T>(V, tok, half), s_red[half], 1 + half);
                if (tok == 0) s_red[half][0] = __float_as_uint(m);
                asm volatile("bar.sync 4, 256;" ::: "memory");
                const float vs = f16_scale(fmaxf(__uint_as_float(s_red[0][0]), __uint_as_float(s_red[1][0])));
                if (tid == 0) s_vs[s] = vs;
                wt *= vs;
                asm volatile("bar.sync 4, 256;" ::: "memory");
            }
            split_row<T>(V, tok, 4 * half, 4 * half + 4, wt, W, W + 16384, W + 32768);
            fence_proxy_async_smem();
            mbar_arrive(&s_w[s]);
        }
    } else if (tid < kSplit + kKeep) {  // ---------------- the state
        float X[StateOf<NB, kKeep>::W];
        load_state<NB, kKeep>(SUM ? StateTile{nullptr, 0, 0, 0} : at.start(w), X);
        char* image = sm + L::image;
        auto keep_sync = [] { asm volatile("bar.sync 3, 256;" ::: "memory"); };
        const bool lead = tid == kSplit;
        for (int ch = 0; ch < chunks; ch++) {
            const int s = ch & 1;
            const uint32_t ph = (ch >> 1) & 1;
            if (!SUM) {
                float sc = 1.0f;
                bool none = false;
                if (kF16<T>) {
                    uint32_t m;
                    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(__float_as_uint(state_max(X))));
                    if ((tid & 31) == 0) s_most[(tid >> 5) & 7] = m;
                }
                if (lead) bulk_wait_read();  // the last image has left
                keep_sync();
                if (kF16<T>) {
                    uint32_t m = 0;
#pragma unroll
                    for (int i = 0; i < 8; i++) m = max(m, s_most[i]);
                    sc = f16_scale(__uint_as_float(m));
                    none = m == 0;
                }
                put_state<T, NB, kKeep, kImage>(image, sc, X);
                fence_proxy_async_smem();
                keep_sync();
                if (lead) {
                    const int64_t at_image = ((b * a.H + h) * ((a.P + PT - 1) / PT) + at.pt) * w.chunks + start_of(ch) / C;
                    bulk_store(static_cast<char*>(at.dir(w).images) + at_image * (kImage * NB * 8192), image, kImage * NB * 8192);
                    bulk_commit();
                    // (a state of zeros gets an infinite scale: what multiplies it then counts for nothing)
                    if (kF16<T>) at.dir(w).image_scale[at_image] = none ? __uint_as_float(0x7f800000u) : sc;
                }
            }
            wait_or_fail(&s_u[s], ph, &s_fail);
            tc_fence_after();
            add_product<NB, kKeep, kParts<T>>(tm + 256 * s, s_all[s], (REV ? a.scale : 1.0f) / (kF16<T> ? s_vs[s] : 1.0f), X);
            tc_fence_before();
            mbar_arrive(&s_free[s]);
        }
        if (SUM) {
            save_state<NB, kKeep>(at.segment(w), X);
        } else if (at.last(w)) {
            save_state<NB, kKeep>(at.whole(w, at.last(w)), X);
        }
        if (lead) bulk_wait_all();
    } else if (tid < kSplit + kKeep + 32) {  // ---------------- weights, tokens 4 lane .. 4 lane + 3
        const int lane = tid & 31;
        float g[4], total = 0.0f;
        auto raw_g = [&](int ch) {
            const int64_t t0 = start_of(ch);
            const int nv = valid(t0);
#pragma unroll
            for (int e = 0; e < 4; e++)
                g[e] = 4 * lane + e < nv ? a.g[a.g_per_head ? h : (b * a.L + t0 + 4 * lane + e) * a.H + h] : 0.0f;
        };
        raw_g(0);
        for (int ch = 0; ch < chunks; ch++) {
            const int s = ch & 1;
            float x[4];
            Two c[4];
#pragma unroll
            for (int e = 0; e < 4; e++) x[e] = clamp_g(g[e]) * kLog2e;
            if (ch + 1 < chunks) raw_g(ch + 1);
            warp_cumsum<4>(x, c);
            const Two cl = {__shfl_sync(kFull, c[3].h, 31), __shfl_sync(kFull, c[3].l, 31)};
            total += cl.h + cl.l;
            if (ch >= 2) wait_or_fail(&s_free[s], ((ch >> 1) & 1) ^ 1, &s_fail);  // the stage's last product is done and read
#pragma unroll
            for (int e = 0; e < 4; e++) s_weight[s][4 * lane + e] = ex2a(REV ? c[e].h + c[e].l : two_diff(cl, c[e]));
            if (lane == 0) s_all[s] = ex2a(cl.h + cl.l);
            mbar_arrive(&s_g[s]);
        }
        if (SUM && lane == 0) w.seg_decay[at.cut * w.plan.K + at.seg] = total / kLog2e;
    } else if ((tid & 31) == 0) {  // ---------------- copies and products
        auto load = [&](int ch) {
            const int s = ch % L::ring, t0 = (int)start_of(ch);
            char* to = sm + s * L::stage;
            mbar_expect_tx(&s_ld[s], (NB + 1) * 16384);
#pragma unroll
            for (int n = 0; n < NB; n++)
                tma_load_4d(to + L::k + n * 16384, REV ? &w.maps.q : &w.maps.k, n * 64, (int)at.hq, t0, (int)b, &s_ld[s]);
            tma_load_4d(to + L::v, REV ? &w.maps.dy : &w.maps.v, (int)at.p0, (int)h, t0, (int)b, &s_ld[s]);
        };
        auto prefetch = [&](int ch) {  // the chunk after those on their way, into the L2 cache
            const int t0 = (int)start_of(ch);
#pragma unroll
            for (int n = 0; n < NB; n++)
                tma_prefetch_4d(REV ? &w.maps.q : &w.maps.k, n * 64, (int)at.hq, t0, (int)b);
            tma_prefetch_4d(REV ? &w.maps.dy : &w.maps.v, (int)at.p0, (int)h, t0, (int)b);
        };
        for (int ch = 0; ch < L::ring - 1 && ch < chunks; ch++) load(ch);
        if (L::ring - 1 < chunks) prefetch(L::ring - 1);
        for (int ch = 0; ch < chunks; ch++) {
            const int s = ch & 1, ahead = ch + L::ring - 1;
            if (ch > 0 && !wait_or_fail(&s_u[s ^ 1], ((ch - 1) >> 1) & 1, &s_fail)) break;
            if (ahead < chunks) load(ahead);  // in the place of chunk ch - 1
            if (ahead + 1 < chunks) prefetch(ahead + 1);
            if (!wait_or_fail(&s_w[s], (ch >> 1) & 1, &s_fail)) break;  // (also: the stage's last product was read)
            tc_fence_after();
            mma_state_wide<T, NB>(tm + 256 * s, sm + (ch % L::ring) * L::stage + L::k, sm + L::w + s * L::parts);
            mma_commit(&s_u[s]);
        }
    }
    uint64_t* const bars[] = {&s_ld[0], &s_ld[1], &s_ld[L::ring - 1], &s_u[0], &s_u[1]};
    end_block(&s_fail, w.status, bars, tm, 512);
}

// seg_state: end state of each segment walked from zero -> the state each
// segment starts from.  One thread per state element; eight segments' states are
// on their way before the first is folded in.
__global__ void __launch_bounds__(256) k_tc_carry(const __grid_constant__ TcWalkArgs w) {
    constexpr int U = 8;
    const int64_t K = w.plan.K, tile = w.a.N * PT, x = (int64_t)blockIdx.x * 256 + threadIdx.x, cut = blockIdx.y;
    if (x >= tile) return;
    Walk at;
    at.place(w, w.plan.whole + cut);
    const bool reverse = at.reverse;
    const StateTile from = at.whole(w, at.dir(w).init);
    float S = from.p && x % PT < from.cols ? from.p[x / PT * from.stride + x % PT] : 0.0f;
    for (int64_t i0 = 0; i0 < K; i0 += U) {
        float own[U], d[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t i = i0 + u, s = cut * K + (reverse ? K - 1 - i : i);
            own[u] = d[u] = 0.0f;
            if (i + 1 < K) {  // the segment walked last has no sum
                own[u] = w.seg_state[s * tile + x];
                d[u] = expf(w.seg_decay[s]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t i = i0 + u, s = cut * K + (reverse ? K - 1 - i : i);
            if (i < K) w.seg_state[s * tile + x] = S;
            S = fmaf(d[u], S, own[u]);
        }
    }
}

template <auto Kernel> cudaError_t go(int threads, int smem, int64_t grid, const TcWalkArgs& w, cudaStream_t st) {
    const cudaError_t e = allow_smem<Kernel>(smem);
    if (e != cudaSuccess) return e;
    Kernel<<<(unsigned)grid, threads, smem, st>>>(w);
    return cudaGetLastError();
}

template <typename T, int NB> cudaError_t fwd_n(const TcWalkArgs& w, cudaStream_t st) {
    return go<k_tc_fwd<T, NB>>(256, FwdSmem<NB>::total, w.plan.blocks(), w, st);
}
template <typename T, int NB> cudaError_t state_n(const TcWalkArgs& w, bool sum, cudaStream_t st) {
    constexpr int smem = StateSmem<NB, kImageParts<kF16<T>, NB>>::total;
    return sum ? go<k_tc_state<T, NB, true>>(kStateThreads, smem, w.plan.cut * (w.plan.K - 1), w, st)
               : go<k_tc_state<T, NB, false>>(kStateThreads, smem, w.plan.blocks(), w, st);
}

}  // namespace

cudaError_t launch_tc_fwd(const TcWalkArgs& w, cudaStream_t st) {
    const bool wide = w.a.N > 64;
    if (w.a.dtype == 1) return wide ? fwd_n<__half, 2>(w, st) : fwd_n<__half, 1>(w, st);
    return wide ? fwd_n<__nv_bfloat16, 2>(w, st) : fwd_n<__nv_bfloat16, 1>(w, st);
}

cudaError_t launch_tc_carry(const TcWalkArgs& w, cudaStream_t st) {
    // cut < 2 * kSms blocks in y
    k_tc_carry<<<dim3((unsigned)ceil_div(w.a.N * PT, 256), (unsigned)w.plan.cut), 256, 0, st>>>(w);
    return cudaGetLastError();
}

cudaError_t launch_tc_state(const TcWalkArgs& w, bool sum, cudaStream_t st) {
    const bool wide = w.a.N > 64;
    if (w.a.dtype == 1) return wide ? state_n<__half, 2>(w, sum, st) : state_n<__half, 1>(w, sum, st);
    return wide ? state_n<__nv_bfloat16, 2>(w, sum, st) : state_n<__nv_bfloat16, 1>(w, sum, st);
}

}  // namespace la
}  // namespace ss
