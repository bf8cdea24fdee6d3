// Linear attention backward on the tensor cores: one chunk of one group of heads
// at a time, from the states before (H) and the state adjoints after (R) every
// chunk.  16-bit io.
//
// Per head (or 64 of its value channels), rows j, columns i >= j, m_ji = e^{c_i - c_j}:
//   S^T = k q^T,  D^T = v dy^T,  P^T = m o S^T,  E^T = scale m o D^T,  W = E^T o S^T (i > j)
//   dv = scale P^T dy + e^{cl - c} (k R)
//   dq += E k + (scale e^c dy) H^T,   dk += E^T q + (e^{cl - c} v) R^T       (over the heads that share q, k)
//   dg_t = sum_{i >= t} a_i + sum_{j < t} (b_j + col_j - row_j) + e^{cl} <R, H>
//     a_i = scale e^{c_i} dy_i . (q_i H),  b_j = e^{cl - c_j} v_j . (k_j R),  col_j, row_i: sums of W over i, j
// dq and dk stay in tensor memory over the heads; q and k are read once for all
// of them.  Roundings to 16 bits: P, E and the scaled dy and v (one rounding of
// each term of a 16-bit output); H and R enter in parts (kImageParts), and dg
// takes everything else in f32.  c_i - c_j inside a run of 32
// tokens is a difference of f32 sums over the run: exact to f32 rounding of the
// run's decay without its resets, which no pair of tokens passes (with them in the sums
// dg was off by 7e-5 where every other token resets).
//
// f16's range needs scales, powers of two that keep every operand's largest value
// near 2^13: P has one, E, the scaled dy and the scaled v share one, H and R come
// with theirs (a zero H or R makes the dy or v that multiplies it zero, so that E alone
// sets the scale).  dq and dk of different heads then cannot add up in tensor memory:
// with f16 a block's work is one head's value tile, and all dq, dk are added up in
// f32 by a kernel of their own.
//
// Measured, bf16, 2 x 4096 tokens, 80 heads that share q and k, N 128, P 64: 229 us
// (DRAM 33 %, tensor cores 33 %, issue 34 %), 34 heads a block of 12 thousand cycles
// each: P, E and W 3000 (the block rows of the first 32 tokens have four times the
// last ones' work, and a warp reaches only its own rows of tensor memory), dv, k R and
// q H 2500, S and D 1000, their reading and the barriers between them the rest.  (With
// the low parts' products of dq and dk before those, 240 us.)  One
// block is all that an SM's tensor and shared memory hold at N = 128.
#include "../simd.cuh"
#include "la_tc.h"
#include "tc.cuh"

namespace ss {
namespace la {
namespace {

constexpr int C = kChunkTc;
constexpr int PT = kTileP;

// x: two places of 32 KB that take turns: v and dy of an iteration, and the low
// parts of its H and R; what is free once k R and q H are done takes the next v
// and dy, what is free once dq and dk are done the next low parts.
template <int NB> struct BwdSmem {
    static constexpr int q = 0, k = q + NB * 16384, x = k + NB * 16384, h = x + 65536, r = h + NB * 8192, e = r + NB * 8192,
                         ds = e + 32768, total = ds + 16384;
};

// Sum over the lanes of x[i] for every i: lane i gets the sum of x[i].
__device__ __forceinline__ float column_sums(float (&x)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; i++) {
            const float keep = up ? x[i + o] : x[i], send = up ? x[i] : x[i + o];
            x[i] = keep + __shfl_xor_sync(kFull, send, o);
        }
    }
    return x[0];
}

// 16 values of a tile's row (units 2 quarter, + 1) as pairs
__device__ __forceinline__ void read_row(void* tile, int row, int quarter, uint32_t (&x)[8]) {
#pragma unroll
    for (int u = 0; u < 2; u++) {
        const uint4 t = *unit(tile, row, 2 * quarter + u);
        x[4 * u] = t.x;
        x[4 * u + 1] = t.y;
        x[4 * u + 2] = t.z;
        x[4 * u + 3] = t.w;
    }
}
__device__ __forceinline__ void write_row(void* tile, int row, int quarter, const uint32_t (&x)[8]) {
#pragma unroll
    for (int u = 0; u < 2; u++)
        *unit(tile, row, 2 * quarter + u) = make_uint4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
}

// A chunk's decays for the compute warps, by runs of 32 tokens; c: log2 decay up
// to and with the token.
struct Decays {
    float c[C];     // c since the run's start, without its resets
    float head[C];  // 2^ of it
    float tail[C];  // 2^(run's end - c)
    float up[C];    // scale 2^c
    float down[C];  // 2^(chunk's end - c)
    float skip[3];  // 2^ from the end of run r to the start of run cb: (r, cb) = (0, 2), (1, 3), (0, 3)
    float all;      // over the chunk
    uint32_t resets[4];  // of each run, a bit a token
};

// Log decays from here on down are resets: e^g is zero in f32.
constexpr float kResetG = -104.0f;

// One warp; g: log decays of tokens 4 lane .. 4 lane + 3.
__device__ __forceinline__ void put_decays(Decays& d, const float (&g)[4], float scale) {
    const int lane = threadIdx.x & 31;
    float x[4];
    Two c[4];
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] = clamp_g(g[e]) * kLog2e;
    warp_cumsum<4>(x, c);
    const auto at = [&](int l) { return Two{__shfl_sync(kFull, c[3].h, l), __shfl_sync(kFull, c[3].l, l)}; };
    const Two end = at(lane | 7), e0 = at(7), e1 = at(15), e2 = at(23), cl = at(31);
    const Two start = lane < 8 ? Two{0.0f, 0.0f} : (lane < 16 ? e0 : (lane < 24 ? e1 : e2));
    float in = 0.0f, own[4];
    uint32_t resets = 0;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const bool reset = g[e] <= kResetG;
        own[e] = in += reset ? 0.0f : x[e];
        resets |= (uint32_t)reset << (4 * (lane & 7) + e);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const float up = __shfl_up_sync(kFull, in, o);
        if ((lane & 7) >= o) in += up;
        resets |= __shfl_xor_sync(kFull, resets, o);
    }
    in = __shfl_up_sync(kFull, in, 1);  // of the lanes before
    if ((lane & 7) == 0) {
        in = 0.0f;
        d.resets[lane >> 3] = resets;
    }
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const int t = 4 * lane + e;
        d.c[t] = in + own[e];
        d.head[t] = ex2a(two_diff(c[e], start));
        d.tail[t] = ex2a(two_diff(end, c[e]));
        d.up[t] = scale * ex2a(c[e].h + c[e].l);
        d.down[t] = ex2a(two_diff(cl, c[e]));
    }
    if (lane == 0) {
        d.skip[0] = ex2a(two_diff(e1, e0));
        d.skip[1] = ex2a(two_diff(e2, e1));
        d.skip[2] = ex2a(two_diff(e2, e0));
        d.all = ex2a(cl.h + cl.l);
    }
}

// Where a block is.  SINGLE: items blockIdx.x, + gridDim.x, ... of one head's value
// tile each.  Else a run of heads (item: the first of them in their group), with the
// value tiles of each.
struct Place {
    int64_t item, end;
    int b, chunk, gq, part, h, h_lo, h_hi, pt, pt_lo, pt_hi;  // part: its row of dq's and dk's parts, -1: the outputs
    int first, last, more;  // of its item's heads and tiles; whether another place follows

    template <bool SINGLE> __device__ void mark() {
        first = h == h_lo && pt == pt_lo;
        last = h + 1 == h_hi && pt + 1 == pt_hi;
        more = !last || item + (SINGLE ? (int64_t)gridDim.x : (int64_t)(h_hi - h_lo)) < end;
    }
    template <bool SINGLE> __device__ void begin(const TcBwdArgs& w, int ptiles) {
        const int rep = (int)(w.a.H / w.a.G), per = SINGLE ? w.splits : rep;
        const int at = (int)(item % per);
        int64_t id = item / per;
        const int64_t left = end - id * per;  // of the run, from the group's first head on
        gq = (int)(id % w.a.G);
        id /= w.a.G;
        chunk = (int)(id % w.chunks);
        b = (int)(id / w.chunks);
        if (SINGLE) {
            h_lo = gq * rep + at / ptiles;
            h_hi = h_lo + 1;
            pt_lo = at % ptiles;
            pt_hi = pt_lo + 1;
            part = w.splits == 1 ? -1 : at * (int)w.a.Bsz + b;
        } else {
            h_lo = gq * rep + at;
            h_hi = gq * rep + (int)min((int64_t)rep, left);
            pt_lo = 0;
            pt_hi = ptiles;
            part = h_hi - h_lo == rep ? -1 : 2 * (int)blockIdx.x + (at == 0);
        }
        h = h_lo;
        pt = pt_lo;
    }
    template <bool SINGLE> __device__ void start(const TcBwdArgs& w, int ptiles) {
        const int64_t all = w.a.Bsz * w.chunks * w.a.G * (SINGLE ? w.splits : (int)(w.a.H / w.a.G));
        item = SINGLE ? (int64_t)blockIdx.x : all * blockIdx.x / gridDim.x;
        end = SINGLE ? all : all * (blockIdx.x + 1) / gridDim.x;
        begin<SINGLE>(w, ptiles);
        mark<SINGLE>();
    }
    template <bool SINGLE> __device__ void step(const TcBwdArgs& w, int ptiles) {  // if more
        if (++pt == pt_hi) {
            pt = pt_lo;
            if (++h == h_hi) {
                item += SINGLE ? (int64_t)gridDim.x : (int64_t)(h_hi - h_lo);
                begin<SINGLE>(w, ptiles);
            }
        }
        mark<SINGLE>();
    }
};

// 16 compute warps (thread: row tok of every tile, a quarter of its columns), a
// warp that issues the products, one that issues the copies (the products' issue
// waits for the tensor cores), and one that makes the decays of the next iteration,
// adds up dg of the last one and sends out what is staged in E.
// Within an iteration (one head's value tile) the products of dq and dk run while
// the compute warps end it and the next one begins.
constexpr int kCompute = 512, kIssue = kCompute, kLoad = kCompute + 32, kHelp = kCompute + 64, kThreads = kCompute + 96;

// Barrier of the compute warps and the issuing warp.
__device__ __forceinline__ void work_sync() { asm volatile("bar.sync 2, 544;" ::: "memory"); }

template <typename T, int NB> __global__ void __launch_bounds__(kThreads, 1) k_tc_bwd(const __grid_constant__ TcBwdArgs w) {
    extern __shared__ __align__(1024) char sm[];
    using L = BwdSmem<NB>;
    constexpr int NP = NB * 64, kImage = kImageParts<kF16<T>, NB>;
    __shared__ Decays s_decays[2];  // of iteration it at it & 1
    __shared__ float s_row[4][C], s_a[4][C], s_b[4][C], s_red[16];
    // copies: v, dy; q, k; states.  Products: S, D; dv, k R, q H; those of the low parts; dq, dk.
    __shared__ __align__(8) uint64_t s_ld, s_kq, s_st, s_m1, s_m2, s_low, s_m3;
    // decays made; the states' low parts and dy read; iteration over; its dg made; E staged; E sent
    __shared__ __align__(8) uint64_t s_dec, s_rh, s_epi, s_dg, s_stage, s_sent;
    __shared__ uint32_t s_tm, s_fail;
    __shared__ uint32_t s_most[kF16<T> ? 4 : 1][16];
    __shared__ Place s_at[3];  // of iteration it at it % 3, the next one's too
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, tok = tid & (C - 1), run = tok >> 5, quarter = tid >> 7;
    char *Q = sm + L::q, *K = sm + L::k, *H = sm + L::h, *R = sm + L::r, *E = sm + L::e, *DS = sm + L::ds;
    const int ptiles = (int)((a.P + PT - 1) / PT);

    if (tid == 0) {
        uint64_t* one[] = {&s_ld, &s_kq, &s_st, &s_m1, &s_m2, &s_low, &s_m3, &s_sent};
        for (uint64_t* b : one) mbar_init(b, 1);
        mbar_init(&s_dec, 32);
        mbar_init(&s_dg, 32);
        mbar_init(&s_rh, kCompute);
        mbar_init(&s_epi, kCompute);
        mbar_init(&s_stage, kCompute);
        s_fail = 0;
        fence_proxy_async_smem();
    }
    if (tid < 32) tmem_alloc(&s_tm, 512);
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tm, my = (uint32_t)(run * 32) << 16;
    // S^T, then P^T and q H in its place; D^T, then dv and k R; dq; dk
    const uint32_t tS = tm, tP = tm, tZ = tm + 64, tD = tm + 128, tV = tm + 128, tF = tm + 192, tQ = tm + 256,
                   tK = tm + 256 + NP;
    auto wait = [&](uint64_t& bar, uint32_t phase) { return wait_or_fail(&bar, phase & 1, &s_fail); };
    auto valid = [&](const Place& p) {
        return (int)max((int64_t)0, min((int64_t)C, row_length(a, p.b) - (int64_t)p.chunk * C));
    };
    auto image_of = [&](const Place& p) { return ((p.b * a.H + p.h) * ptiles + p.pt) * w.chunks + p.chunk; };
    // rounds through E at an item's end (dv has one at every iteration's): bf16 tiles of dq and dk, or f32 tiles
    auto qk_rounds = [](const Place& p) { return p.part < 0 ? NB : 2 * NB; };
    Place at;  // the other warps
    if (tid >= kCompute) at.start<kF16<T>>(w, ptiles);

    if (tid >= kHelp) {  // ---------------- the helping warp
        const bool lead = lane == 0;
        auto put_dg = [&](const Place& at) {  // of its head (f16: its tile's part), tokens 4 lane .. 4 lane + 3
            if (at.pt + 1 < at.pt_hi) return;
            const int64_t t0 = (int64_t)at.chunk * C;
            const int nv = valid(at);
            float sum = 0.0f, av[4], bv[4];
#pragma unroll
            for (int u = 0; u < 16; u++) sum += s_red[u];
            float A = 0.0f, B = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int t = 4 * lane + e;
                av[e] = (s_a[0][t] + s_a[1][t]) + (s_a[2][t] + s_a[3][t]);
                bv[e] = (s_b[0][t] + s_b[1][t]) + (s_b[2][t] + s_b[3][t]);
                A += av[e];
                B += bv[e];
            }
            float suf = A, pre = B;  // inclusive over lanes, from the right and from the left
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float x = __shfl_down_sync(kFull, suf, o), y = __shfl_up_sync(kFull, pre, o);
                if (lane + o < 32) suf += x;
                if (lane >= o) pre += y;
            }
            pre -= B;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int64_t t = 4 * lane + e;
                if (t0 + t < a.L) w.dg[((at.pt_lo * a.Bsz + at.b) * a.L + t0 + t) * a.H + at.h] = t < nv ? suf + pre + sum : 0.0f;
                suf -= av[e];
                pre += bv[e];
            }
        };
        auto raw_g = [&](const Place& p, float (&g)[4]) {
            const int nv = valid(p);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int t = 4 * lane + e;
                g[e] = t < nv ? a.g[a.g_per_head ? (int64_t)p.h : ((p.b * a.L + (int64_t)p.chunk * C + t) * a.H + p.h)] : 0.0f;
            }
        };
        uint32_t round = 0;
        // sends what the compute warps staged in E (one tile or two), zeros past the row's length: zero rows times a
        // state or an operand that is not finite are not zero (as selects in the compute warps: 18 us more of 383)
        int lo, hi;  // the chunk's tokens past the length
        auto send = [&](int tiles, auto store) {
            wait(s_stage, round++);
            if (lo < hi) {
                for (int k = 0; k < tiles; k++)
#pragma unroll 4
                    for (int i = lo * 8 + lane; i < hi * 8; i += 32)
                        *reinterpret_cast<uint4*>(E + k * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lead) {
                if (!s_fail) store();
                bulk_commit();
                bulk_wait_read();
                mbar_arrive(&s_sent);
            }
            __syncwarp();
        };
        float g[4];
        raw_g(at, g);
        if (lead) s_at[0] = at;
        put_decays(s_decays[0], g, a.scale);
        mbar_arrive(&s_dec);
        for (uint32_t it = 0;; it++) {
            Place next = at;
            if (at.more) {
                next.step<kF16<T>>(w, ptiles);
                raw_g(next, g);
                // (the last iteration is over: nothing reads that place and those decays any more)
                if (lead) s_at[(it + 1) % 3] = next;
                put_decays(s_decays[(it + 1) & 1], g, a.scale);
                mbar_arrive(&s_dec);
            }
            lo = valid(at);
            hi = (int)min((int64_t)C, a.L - (int64_t)at.chunk * C);
            wait(s_epi, it);
            put_dg(at);
            mbar_arrive(&s_dg);
            send(1, [&] { tma_store_4d(&w.maps.dv, E, at.pt * PT, at.h, at.chunk * C, at.b); });
            if (at.last)
                for (int k = 0; k < qk_rounds(at); k++)
                    send(2, [&] {
                        const int t0 = at.chunk * C;
                        if (at.part < 0) {  // NB == 1: dq and dk; NB == 2: both halves of one of them
                            tma_store_4d(NB == 1 || k == 0 ? &w.maps.dq : &w.maps.dk, E, 0, at.gq, t0, at.b);
                            if (NB == 1) tma_store_4d(&w.maps.dk, E + 16384, 0, at.gq, t0, at.b);
                            else tma_store_4d(k == 0 ? &w.maps.dq : &w.maps.dk, E + 16384, 64, at.gq, t0, at.b);
                        } else {  // 64 columns of dq or dk, 32 a tile
                            const CUtensorMap* map = k < NB ? &w.maps.dq_part : &w.maps.dk_part;
                            const int n = (k % NB) * 64, g = kF16<T> ? at.gq : 0, t = kF16<T> ? t0 : 0;
                            tma_store_4d(map, E, n, g, t, at.part);
                            tma_store_4d(map, E + 16384, n + 32, g, t, at.part);
                        }
                    });
            if (!at.more) break;
            at = next;
        }
        if (lead) bulk_wait_all();
    } else if (tid >= kLoad) {  // ---------------- the loading warp
        if (lane == 0) {
            auto load_kq = [&](const Place& p) {
                mbar_expect_tx(&s_kq, 2 * NB * 16384);
#pragma unroll
                for (int n = 0; n < NB; n++) {
                    tma_load_4d(K + n * 16384, &w.maps.k, n * 64, p.gq, p.chunk * C, p.b, &s_kq);
                    tma_load_4d(Q + n * 16384, &w.maps.q, n * 64, p.gq, p.chunk * C, p.b, &s_kq);
                }
            };
            auto load_v = [&](const Place& p, uint32_t it) {
                char* to = sm + L::x + (it & 1) * 32768;
                mbar_expect_tx(&s_ld, 32768);
                tma_load_4d(to, &w.maps.v, p.pt * PT, p.h, p.chunk * C, p.b, &s_ld);
                tma_load_4d(to + 16384, &w.maps.dy, p.pt * PT, p.h, p.chunk * C, p.b, &s_ld);
            };
            constexpr int part = NB * 8192, low = (kImage - 1) * part;
            auto load_states = [&](const Place& p, uint32_t it) {
                char* to = sm + L::x + ((it & 1) ^ 1) * 32768;
                const char *hs = static_cast<const char*>(w.before) + image_of(p) * kImage * part,
                           *rs = static_cast<const char*>(w.after) + image_of(p) * kImage * part;
                mbar_expect_tx(&s_st, 2 * kImage * part);
                bulk_load(H, hs, part, &s_st);
                bulk_load(R, rs, part, &s_st);
                bulk_load(to, hs + part, low, &s_st);
                bulk_load(to + 16384, rs + part, low, &s_st);
            };
            load_kq(at);
            load_v(at, 0);
            load_states(at, 0);
            auto prefetch = [&](const Place& p) {
                tma_prefetch_4d(&w.maps.v, p.pt * PT, p.h, p.chunk * C, p.b);
                tma_prefetch_4d(&w.maps.dy, p.pt * PT, p.h, p.chunk * C, p.b);
                bulk_prefetch(static_cast<const char*>(w.before) + image_of(p) * kImage * part, kImage * part);
                bulk_prefetch(static_cast<const char*>(w.after) + image_of(p) * kImage * part, kImage * part);
            };
            for (uint32_t it = 0; at.more; it++) {
                at.step<kF16<T>>(w, ptiles);
                prefetch(at);
                wait(s_rh, it);
                if (wait(s_low, it)) load_v(at, it + 1);
                if (wait(s_m3, it)) {
                    if (at.first) load_kq(at);
                    load_states(at, it + 1);
                }
            }
        }
    } else if (tid >= kIssue) {  // ---------------- the issuing warp
        const bool lead = lane == 0;
        uint32_t kq = 0, it = 0;
        for (;; it++) {
            const uint32_t ph = it & 1;
            char *V = sm + L::x + ph * 32768, *DY = V + 16384, *HL = sm + L::x + (ph ^ 1) * 32768, *RL = HL + 16384;
            const bool first = at.first;
            wait(s_ld, it);
            if (first) wait(s_kq, kq++);
            work_sync();  // A: tiles ready, the last iteration's accumulators read
            if (lead && !s_fail) {
                tc_fence_after();
                constexpr uint32_t d = mma_desc<T>(128, 128, false, false);
#pragma unroll
                for (int s = 0; s < 4 * NB; s++) {
                    const uint32_t o = (s >> 2) * 16384 + (s & 3) * 32;
                    mma(tS, smem_desc(smem_addr(K) + o), smem_desc(smem_addr(Q) + o), d, s > 0);
                }
#pragma unroll
                for (int s = 0; s < 4; s++)
                    mma(tD, smem_desc(smem_addr(V) + s * 32), smem_desc(smem_addr(DY) + s * 32), d, s > 0);
                mma_commit(&s_m1);
            }
            __syncwarp();
            work_sync();  // S and D have been read
            wait(s_st, it);
            work_sync();  // B: P, E and the scaled tiles are there
            if (lead && !s_fail) {
                tc_fence_after();
                constexpr uint32_t dV = mma_desc<T>(128, PT, false, true), dQ = mma_desc<T>(128, NP, true, true),
                                   dQs = mma_desc<T>(128, NP, false, false), dK = mma_desc<T>(128, NP, false, true);
#pragma unroll
                for (int s = 0; s < C / 16; s++) mma_ts(tV, tP + 8 * s, smem_desc(smem_addr(DY) + s * 2048), dV, s > 0);
#pragma unroll
                for (int s = 0; s < 4 * NB * kImage; s++) {  // k R and q H, all parts
                    const int n = s % (4 * NB), low = (s / (4 * NB) - 1) * NB * 8192;
                    const uint32_t o = (n >> 2) * 16384 + (n & 3) * 32;
                    mma(tF, smem_desc(smem_addr(K) + o), smem_desc(smem_addr(low < 0 ? R : RL + low) + n * 2048), dV, s > 0);
                    mma(tZ, smem_desc(smem_addr(Q) + o), smem_desc(smem_addr(low < 0 ? H : HL + low) + n * 2048), dV, s > 0);
                }
                mma_commit(&s_m2);
#pragma unroll
                for (int s = 0; s < PT / 16; s++) {  // the second parts in dq and dk: one rounding less (of dy and v only)
                    mma(tQ, smem_desc(smem_addr(DS) + s * 32), smem_desc(smem_addr(HL) + s * 32), dQs, !first || s > 0);
                    mma(tK, smem_desc(smem_addr(V) + s * 32), smem_desc(smem_addr(RL) + s * 32), dQs, !first || s > 0);
                }
                mma_commit(&s_low);
#pragma unroll
                for (int s = 0; s < C / 16; s++) {
                    mma(tQ, smem_desc(smem_addr(E) + s * 2048, 16384), smem_desc(smem_addr(K) + s * 2048, 16384), dQ, true);
                    mma(tK, smem_desc(smem_addr(E) + (s >> 2) * 16384 + (s & 3) * 32), smem_desc(smem_addr(Q) + s * 2048, 16384),
                        dK, true);
                }
#pragma unroll
                for (int s = 0; s < PT / 16; s++) {
                    mma(tQ, smem_desc(smem_addr(DS) + s * 32), smem_desc(smem_addr(H) + s * 32), dQs, true);
                    mma(tK, smem_desc(smem_addr(V) + s * 32), smem_desc(smem_addr(R) + s * 32), dQs, true);
                }
                mma_commit(&s_m3);
            }
            __syncwarp();
            if (!at.more) break;
            at.step<kF16<T>>(w, ptiles);
        }
        wait(s_m3, it);
    } else {  // ---------------- the compute warps
        uint32_t round = 0;
        auto stage = [&](auto fill) {  // a round through E: what was there has been sent
            if (round > 0) wait(s_sent, round - 1);
            round++;
            fill();
            fence_proxy_async_smem();
            mbar_arrive(&s_stage);
        };
        // what an iteration leaves: dv; after an item's last one, dq and dk of the group (or of a part of its heads)
        auto put_out = [&](const Place& at, const uint32_t (&dv)[8], float kap) {
            stage([&] { write_row(E, tok, quarter, dv); });
            if (!at.last) return;
            for (int k = 0; k < qk_rounds(at); k++)
                stage([&] {
                    if (at.part < 0) {
#pragma unroll
                        for (int c = 0; c < 2; c++) {  // 16 columns of a tile each: NB == 1: of dq, dk; NB == 2: of two tiles
                            const uint32_t from = NB == 1 ? (c == 0 ? tQ : tK) : (k == 0 ? tQ : tK) + 64 * c;
                            float x[16];
                            uint32_t r[8];
                            tmem_ld16(from + my + 16 * quarter, x);
#pragma unroll
                            for (int i = 0; i < 8; i++) r[i] = kF16<T> ? pack2<T>(x[2 * i] / kap, x[2 * i + 1] / kap) : pack2<T>(x[2 * i], x[2 * i + 1]);
                            write_row(E + c * 16384, tok, quarter, r);
                        }
                    } else {
                        float x[16];
                        tmem_ld16((k < NB ? tQ : tK) + 64 * (k % NB) + my + 16 * quarter, x);
#pragma unroll
                        for (int u = 0; u < 4; u++) {
                            float4 f = make_float4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
                            if (kF16<T>) f = make_float4(f.x / kap, f.y / kap, f.z / kap, f.w / kap);
                            *reinterpret_cast<float4*>(unit(E + (quarter >> 1) * 16384, tok, (quarter & 1) * 4 + u)) = f;
                        }
                    }
                });
            tc_fence_before();
        };
        float through = 0.0f, kap_last = 1.0f;
        uint32_t dv[8], kq = 0, it = 0;
        for (;; it++) {
            const uint32_t ph = it & 1;
            char *V = sm + L::x + ph * 32768, *DY = V + 16384, *HL = sm + L::x + (ph ^ 1) * 32768, *RL = HL + 16384;
            wait(s_dec, it);
            const Place& at = s_at[it % 3];
            const Decays& dec = s_decays[ph];
            const int64_t t0 = (int64_t)at.chunk * C;
            const int nv = valid(at);
            bool ok = wait(s_ld, it);
            if (at.first) ok = wait(s_kq, kq++) && ok;
            if (ok && tok >= nv && t0 + tok < a.L) {  // tokens beyond the row's length
                const uint32_t zero[8] = {};
                write_row(V, tok, quarter, zero);
                write_row(DY, tok, quarter, zero);
                if (at.first)
#pragma unroll
                    for (int n = 0; n < NB; n++) {
                        write_row(Q + n * 16384, tok, quarter, zero);
                        write_row(K + n * 16384, tok, quarter, zero);
                    }
                fence_proxy_async_smem();
            }
            tc_fence_before();
            work_sync();  // A
            if (it > 0) {  // the last products have read E, the scaled dy and v
                wait(s_m3, it - 1);
                tc_fence_after();
                put_out(s_at[(it + 2) % 3], dv, kap_last);
            }
            const float down = dec.down[tok];
            uint32_t vr[8];
            read_row(V, tok, quarter, vr);
            auto put_ds = [&](float f) {  // f dy
                uint32_t x[8];
                read_row(DY, tok, quarter, x);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float2 y = mul2(unpack2<T>(x[i]), splat2(f));
                    x[i] = pack2<T>(y.x, y.y);
                }
                write_row(DS, tok, quarter, x);
            };
            auto put_v = [&](float f) {  // f v, in v's place
                uint32_t x[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float2 y = mul2(unpack2<T>(vr[i]), splat2(f));
                    x[i] = pack2<T>(y.x, y.y);
                }
                write_row(V, tok, quarter, x);
            };
            if (!kF16<T>) put_ds(dec.up[tok]);
            wait(s_m1, it);
            tc_fence_after();
            if (!kF16<T>) put_v(down);
            // P, E and W by 32 x 32 blocks: rows of `run`, columns of `quarter`.  W keeps its diagonal: it is in a
            // row's sum and in a column's, which dg subtracts
            uint32_t pr[16], er[16];
            float col = 0.0f, ih = 1.0f, ir = 1.0f, kap = 1.0f, ps = 1.0f;
            const int cb = quarter;
            // the block: S, D from tensor memory; use(i, P, E, S) for its column pairs
            auto block = [&](auto use) {
                float s[32], d[32];
                tmem_ld32(tS + my + 32 * cb, s);
                tmem_ld32(tD + my + 32 * cb, d);
                const float2 f = splat2(cb > run ? dec.tail[tok] * (cb == run + 1 ? 1.0f : dec.skip[cb - 2 + (cb - run == 3 ? 1 : 0)])
                                                 : -dec.c[tok]);
                if (cb > run) {
                    const float2 fs = mul2(f, splat2(a.scale));
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 t = *reinterpret_cast<const float2*>(&dec.head[32 * cb + j]);
                        const float2 sv = make_float2(s[j], s[j + 1]);
                        use(j, mul2(mul2(f, t), sv), mul2(mul2(fs, t), make_float2(d[j], d[j + 1])), sv);
                    }
                } else {
                    if (dec.resets[run]) {  // nothing passes one
                        const uint32_t after = dec.resets[run] & ~((2u << lane) - 1);
                        const int stop = after ? __ffs(after) - 1 : 32;
#pragma unroll
                        for (int j = 0; j < 32; j++)
                            if (j >= stop) s[j] = d[j] = 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 c = add2(*reinterpret_cast<const float2*>(&dec.c[32 * cb + j]), f);
                        const float2 m = make_float2(j >= lane ? ex2a(c.x) : 0.0f, j + 1 >= lane ? ex2a(c.y) : 0.0f);
                        const float2 sv = make_float2(s[j], s[j + 1]);
                        use(j, mul2(m, sv), mul2(mul2(m, splat2(a.scale)), make_float2(d[j], d[j + 1])), sv);
                    }
                }
            };
            if (cb >= run) {
                float wv[32];
                float2 sum = splat2(0.0f), most = splat2(0.0f);
                block([&](int j, float2 p, float2 e, float2 sv) {
                    const float2 x = mul2(e, sv);
                    sum = add2(sum, x);
                    wv[j] = x.x;
                    wv[j + 1] = x.y;
                    if (kF16<T>) {
                        most.x = fmaxf(most.x, fmaxf(fabsf(p.x), fabsf(p.y)));
                        most.y = fmaxf(most.y, fmaxf(fabsf(e.x), fabsf(e.y)));
                    } else {
                        pr[j / 2] = pack2<T>(p.x, p.y);
                        er[j / 2] = pack2<T>(e.x, e.y);
                    }
                });
                col = sum.x + sum.y;
                s_row[run][32 * cb + lane] = column_sums(wv);
                if (kF16<T>) {
                    ps = most.x;
                    kap = most.y;
                }
            } else {
                if (kF16<T>) ps = kap = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; i++) pr[i] = er[i] = 0;
            }
            if constexpr (kF16<T>) {
                // the scales: the block's largest P, E, scaled dy and scaled v
                float md = 0.0f, mv = 0.0f;
                uint32_t x[8];
                read_row(DY, tok, quarter, x);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float2 y = unpack2<T>(x[i]), v = unpack2<T>(vr[i]);
                    md = fmaxf(md, fmaxf(fabsf(y.x), fabsf(y.y)));
                    mv = fmaxf(mv, fmaxf(fabsf(v.x), fabsf(v.y)));
                }
                const int64_t image = image_of(at);
                ih = 1.0f / w.before_scale[image];
                ir = 1.0f / w.after_scale[image];
                const float most[4] = {ps, kap, md * fabsf(dec.up[tok]) * ih, mv * down * ir};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    uint32_t m;
                    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(__float_as_uint(most[i])));
                    if (lane == 0) s_most[i][tid >> 5] = m;
                }
                asm volatile("bar.sync 1, 512;" ::: "memory");
                uint32_t mp = 0, mk = 0;
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    mp = max(mp, s_most[0][i]);
                    mk = max(mk, max(s_most[1][i], max(s_most[2][i], s_most[3][i])));
                }
                ps = f16_scale(__uint_as_float(mp));
                kap = f16_scale(__uint_as_float(mk));
                put_ds(dec.up[tok] * ih * kap);
                put_v(down * ir * kap);
                if (cb >= run)
                    block([&](int j, float2 p, float2 e, float2) {
                        p = mul2(p, splat2(ps));
                        e = mul2(e, splat2(kap));
                        pr[j / 2] = pack2<T>(p.x, p.y);
                        er[j / 2] = pack2<T>(e.x, e.y);
                    });
            }
            if (round > 0) wait(s_sent, round - 1);
            // E: row j, columns 32 cb .. + 31 of two 64-column tiles
#pragma unroll
            for (int u = 0; u < 4; u++)
                *unit(E + (cb >> 1) * 16384, tok, (cb & 1) * 4 + u) = make_uint4(er[4 * u], er[4 * u + 1], er[4 * u + 2], er[4 * u + 3]);
            tc_fence_before();
            work_sync();  // S and D have been read
            tc_fence_after();
            tmem_st16(tP + my + 16 * cb, pr);
            tmem_wait_st();
            tc_fence_before();
            fence_proxy_async_smem();
            wait(s_st, it);
            if (it > 0) wait(s_dg, it - 1);  // what dg reads may be written again
            work_sync();                     // B
            // <R, H> of this tile: rows n of both
            if (at.pt == at.pt_lo) through = 0.0f;
            if (tok < NP) {
                uint32_t h[8], r[8];
                float2 hv[8], rv[8], acc = splat2(0.0f);
#pragma unroll
                for (int p = 0; p < kImage; p++) {
                    read_row(p == 0 ? H : HL + (p - 1) * NB * 8192, tok, quarter, h);
                    read_row(p == 0 ? R : RL + (p - 1) * NB * 8192, tok, quarter, r);
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        hv[i] = p == 0 ? unpack2<T>(h[i]) : add2(hv[i], unpack2<T>(h[i]));
                        rv[i] = p == 0 ? unpack2<T>(r[i]) : add2(rv[i], unpack2<T>(r[i]));
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; i++) acc = fma2(hv[i], rv[i], acc);
                through += acc.x + acc.y;
            }
            float th = through;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) th += __shfl_xor_sync(kFull, th, o);
            if (lane == 0) s_red[tid >> 5] = th * (dec.all * ih * ir);
            uint32_t dyr[8];
            read_row(DY, tok, quarter, dyr);
            mbar_arrive(&s_rh);
            wait(s_m2, it);
            tc_fence_after();
            {
                float f[16], x[16], zz[16];
                tmem_ld16(tF + my + 16 * quarter, f);
                tmem_ld16(tV + my + 16 * quarter, x);
                tmem_ld16(tZ + my + 16 * quarter, zz);
                float2 b = make_float2(0.0f, 0.0f), z = make_float2(0.0f, 0.0f);
                const float fv = a.scale / ps, fr = down * ir;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float2 y = mul2(splat2(fr), make_float2(f[2 * i], f[2 * i + 1]));
                    b = fma2(y, unpack2<T>(vr[i]), b);
                    z = fma2(make_float2(zz[2 * i], zz[2 * i + 1]), unpack2<T>(dyr[i]), z);
                    const float2 o = fma2(splat2(fv), make_float2(x[2 * i], x[2 * i + 1]), y);
                    dv[i] = pack2<T>(o.x, o.y);
                }
                float sa = dec.up[tok] * ih * (z.x + z.y), sb = b.x + b.y + col;
                if (quarter <= run) sb -= s_row[quarter][tok];  // row_i, one row block each
                if (at.pt > at.pt_lo) {
                    sa += s_a[quarter][tok];
                    sb += s_b[quarter][tok];
                }
                s_a[quarter][tok] = sa;
                s_b[quarter][tok] = sb;
            }
            kap_last = kap;
            const bool more = at.more;
            mbar_arrive(&s_epi);
            if (!more) break;
        }
        wait(s_m3, it);
        tc_fence_after();
        put_out(s_at[it % 3], dv, kap_last);
    }
    uint64_t* const bars[] = {&s_ld, &s_kq, &s_st, &s_m1, &s_m2, &s_low, &s_m3};
    end_block(&s_fail, w.status, bars, tm, 512);
}

// dq and dk of the groups that the blocks' runs cut: sums of their parts in the
// runs' order.  Block x of `runs` - 1: the group that run x cuts and holds the start of.
// Bound by memory (13 us for 28 MB of parts, most of them in the L2 cache).
__global__ void __launch_bounds__(256) k_tc_join(const __grid_constant__ TcBwdArgs w, int runs) {
    __shared__ int s_parts, s_t0;  // parts after the first (-1: nothing to do); the chunk's first token
    __shared__ int64_t s_out;      // its place in dq and dk
    const Args& a = w.a;
    if (threadIdx.x == 0) {
        const int64_t rep = a.H / a.G, all = a.Bsz * w.chunks * a.H;
        auto begin = [&](int64_t x) { return all * x / runs; };
        int64_t x = blockIdx.x, id = begin(x + 1) / rep;
        const int64_t first = id * rep, end = first + rep;
        int parts = -1;
        if (begin(x + 1) > first && begin(x) <= first) {
            parts = 0;
            while (begin(++x) < end) parts++;
        }
        s_parts = parts;
        const int64_t gq = id % a.G, b = id / a.G / w.chunks;
        s_t0 = (int)(id / a.G % w.chunks) * C;
        s_out = ((b * a.L + s_t0) * a.G + gq) * a.N;
    }
    __syncthreads();
    const int parts = s_parts, N = (int)a.N;
    const int e = (blockIdx.y * 256 + threadIdx.x) * 4, t = e / N;
    if (parts < 0 || t >= C || s_t0 + t >= a.L) return;
    const int64_t size = C * N;
    const float* part = (blockIdx.z ? w.dk_part : w.dq_part) + 2 * (int64_t)blockIdx.x * size + e;
    float4 s = *reinterpret_cast<const float4*>(part + size);
    for (int u0 = 1; u0 <= parts; u0 += 4) {  // four parts on their way at a time
        float4 y[4];
#pragma unroll
        for (int u = 0; u < 4; u++)
            y[u] = u0 + u <= parts ? *reinterpret_cast<const float4*>(part + 2 * (u0 + u) * size) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int u = 0; u < 4; u++) s = {s.x + y[u].x, s.y + y[u].y, s.z + y[u].z, s.w + y[u].w};
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(blockIdx.z ? w.dk : w.dq) + s_out + (int64_t)t * a.G * N + e % N;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack2<__nv_bfloat16>(s.x, s.y), pack2<__nv_bfloat16>(s.z, s.w));
}

// A block one part of which is long over when another's wait, on a barrier that nothing
// completes, runs out.
__global__ void __launch_bounds__(64, 1) k_late_timeout(int* status, uint64_t limit_ns) {
    __shared__ __align__(8) uint64_t s_bar;
    __shared__ uint32_t s_tm, s_fail;
    if (threadIdx.x == 0) {
        mbar_init(&s_bar, 1);
        s_fail = 0;
        fence_proxy_async_smem();
    }
    if (threadIdx.x < 32) tmem_alloc(&s_tm, 32);
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x >= 32) wait_or_fail(&s_bar, 0, &s_fail, limit_ns);
    uint64_t* const bars[] = {&s_bar};
    end_block(&s_fail, status, bars, s_tm, 32);
}

template <typename T, int NB> cudaError_t bwd_n(const TcBwdArgs& w, cudaStream_t st) {
    constexpr int smem = BwdSmem<NB>::total;
    cudaError_t e = allow_smem<k_tc_bwd<T, NB>>(smem);
    if (e != cudaSuccess) return e;
    const int64_t rep = w.a.H / w.a.G, all = w.a.Bsz * w.chunks * w.a.G * (kF16<T> ? w.splits : rep), blocks = tc_bwd_blocks(all);
    k_tc_bwd<T, NB><<<(unsigned)blocks, kThreads, smem, st>>>(w);
    e = cudaGetLastError();
    // (groups of one head, and equal runs of whole groups, leave nothing to join)
    if (kF16<T> || e != cudaSuccess || rep == 1 || (all % blocks == 0 && all / blocks % rep == 0)) return e;
    k_tc_join<<<dim3((unsigned)blocks - 1, (unsigned)ceil_div(C * w.a.N, 1024), 2), 256, 0, st>>>(w, (int)blocks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_late_timeout(int* status, uint64_t limit_ns, cudaStream_t st) {
    k_late_timeout<<<1, 64, 0, st>>>(status, limit_ns);
    return cudaGetLastError();
}

cudaError_t launch_tc_bwd(const TcBwdArgs& w, cudaStream_t st) {
    if (w.a.dtype == 1) return w.a.N > 64 ? bwd_n<__half, 2>(w, st) : bwd_n<__half, 1>(w, st);
    return w.a.N > 64 ? bwd_n<__nv_bfloat16, 2>(w, st) : bwd_n<__nv_bfloat16, 1>(w, st);
}

}  // namespace la
}  // namespace ss
