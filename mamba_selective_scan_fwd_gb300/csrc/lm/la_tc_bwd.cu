// Linear attention backward on the tensor cores: one chunk of one group of heads
// at a time, from the states before (H) and the state adjoints after (R) every
// chunk.  bf16 io.
//
// Per head (or 64 of its value channels), rows j, columns i >= j, m_ji = e^{c_i - c_j}:
//   S^T = k q^T,  D^T = v dy^T,  P^T = m o S^T,  E^T = scale m o D^T,  W = E^T o S^T (i > j)
//   dv = scale P^T dy + e^{cl - c} (k R)
//   dq += E k + (scale e^c dy) H^T,   dk += E^T q + (e^{cl - c} v) R^T       (over the heads that share q, k)
//   dg_t = sum_{i >= t} a_i + sum_{j < t} (b_j + col_j - row_j) + e^{cl} <R, H>
//     a_i = scale e^{c_i} dy_i . (q_i H),  b_j = e^{cl - c_j} v_j . (k_j R),  col_j, row_i: sums of W over i, j
// dq and dk stay in tensor memory over the heads; q and k are read once for all
// of them.  Roundings to 16 bits: P, E, the scaled dy and v, and H and R as
// operands of dq and dk (outputs of 16 bits); dg takes k R and q H with both
// parts of R and H and everything else in f32.
#include "../simd.cuh"
#include "la_tc.h"
#include "tc.cuh"

namespace ss {
namespace la {
namespace {

constexpr int C = kChunkTc;
constexpr int PT = kTileP;

template <int NB> struct BwdSmem {
    static constexpr int q = 0, k = q + NB * 16384, v = k + NB * 16384, dy = v + 16384, h = dy + 16384,
                         r = h + 2 * NB * 8192, e = r + 2 * NB * 8192, ds = e + 32768, total = ds + 16384;
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

// 32 values of a tile's row (units 4 half .. 4 half + 3) as pairs
__device__ __forceinline__ void read_row(void* tile, int row, int half, uint32_t (&x)[16]) {
#pragma unroll
    for (int u = 0; u < 4; u++) {
        const uint4 t = *unit(tile, row, 4 * half + u);
        x[4 * u] = t.x;
        x[4 * u + 1] = t.y;
        x[4 * u + 2] = t.z;
        x[4 * u + 3] = t.w;
    }
}
__device__ __forceinline__ void write_row(void* tile, int row, int half, const uint32_t (&x)[16]) {
#pragma unroll
    for (int u = 0; u < 4; u++)
        *unit(tile, row, 4 * half + u) = make_uint4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
}

template <typename T, int NB> __global__ void __launch_bounds__(256, 1) k_tc_bwd(const __grid_constant__ TcBwdArgs w) {
    extern __shared__ __align__(1024) char sm[];
    using L = BwdSmem<NB>;
    constexpr int NP = NB * 64;
    __shared__ __align__(16) Two s_c[C];
    __shared__ __align__(16) float s_head[C];
    __shared__ float s_row[4][C], s_a[2][C], s_b[2][C], s_red[8];
    __shared__ Two s_end[4];
    // copies: v, dy (and q, k); states.  Products: S, D; dv, k R, q H; dq, dk
    __shared__ __align__(8) uint64_t s_ld, s_st, s_m1, s_m2, s_m3;
    __shared__ uint32_t s_tm;
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, tok = tid & (C - 1), run = tok >> 5, half = tid >> 7;
    char *Q = sm + L::q, *K = sm + L::k, *V = sm + L::v, *DY = sm + L::dy, *H = sm + L::h, *R = sm + L::r, *E = sm + L::e,
         *DS = sm + L::ds;
    const int64_t rep = a.H / a.G, ptiles = (a.P + PT - 1) / PT;
    const int64_t items = a.Bsz * w.chunks * a.G * w.splits;

    if (tid == 0) {
        mbar_init(&s_ld, 1);
        mbar_init(&s_st, 1);
        mbar_init(&s_m1, 1);
        mbar_init(&s_m2, 1);
        mbar_init(&s_m3, 1);
        fence_proxy_async_smem();
    }
    if (tid < 32) tmem_alloc(&s_tm, 512);
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tm, my = (uint32_t)(run * 32) << 16;
    // S^T, then P^T and q H in its place; D^T, then dv and k R; dq; dk
    const uint32_t tS = tm, tP = tm, tZ = tm + 64, tD = tm + 128, tV = tm + 128, tF = tm + 192, tQ = tm + 256,
                   tK = tm + 256 + NP;

    // A block's work: items blockIdx.x, + gridDim.x, ...; in each the heads h_lo .. h_hi - 1, their value tiles
    struct Place {
        int64_t item, b, chunk, gq, split, h, h_lo, h_hi, pt;
    };
    auto begin = [&](Place& p) {
        int64_t id = p.item;
        p.split = id % w.splits;
        id /= w.splits;
        p.gq = id % a.G;
        id /= a.G;
        p.chunk = id % w.chunks;
        p.b = id / w.chunks;
        p.h_lo = p.gq * rep + rep * p.split / w.splits;
        p.h_hi = p.gq * rep + rep * (p.split + 1) / w.splits;
        p.h = p.h_lo;
        p.pt = 0;
    };
    auto step = [&](Place& p) {  // the next place; false past the last
        if (++p.pt < ptiles) return true;
        p.pt = 0;
        if (++p.h < p.h_hi) return true;
        p.item += gridDim.x;
        if (p.item >= items) return false;
        begin(p);
        return true;
    };
    auto load = [&](const Place& p) {
        const int t0 = (int)(p.chunk * C);
        const bool first = p.h == p.h_lo && p.pt == 0;
        mbar_expect_tx(&s_ld, (first ? 2 * NB + 2 : 2) * 16384);
        if (first)
#pragma unroll
            for (int n = 0; n < NB; n++) {
                tma_load_4d(K + n * 16384, &w.maps.k, n * 64, (int)p.gq, t0, (int)p.b, &s_ld);
                tma_load_4d(Q + n * 16384, &w.maps.q, n * 64, (int)p.gq, t0, (int)p.b, &s_ld);
            }
        tma_load_4d(V, &w.maps.v, (int)(p.pt * PT), (int)p.h, t0, (int)p.b, &s_ld);
        tma_load_4d(DY, &w.maps.dy, (int)(p.pt * PT), (int)p.h, t0, (int)p.b, &s_ld);
        constexpr int bytes = 2 * NB * 8192;
        const int64_t image = ((p.b * a.H + p.h) * ptiles + p.pt) * w.chunks + p.chunk;
        mbar_expect_tx(&s_st, 2 * bytes);
        bulk_load(H, static_cast<const char*>(w.before) + image * bytes, bytes, &s_st);
        bulk_load(R, static_cast<const char*>(w.after) + image * bytes, bytes, &s_st);
    };
    Place at;
    at.item = blockIdx.x;
    begin(at);
    if (tid == 0) load(at);
    auto valid = [&](const Place& p) {
        return (int)max((int64_t)0, min((int64_t)C, row_length(a, p.b) - p.chunk * C));
    };
    auto load_g = [&](const Place& p, int nv) {
        return tok < nv ? log_decay(a, p.b, p.chunk * C + tok, p.h) * kLog2e : 0.0f;
    };
    int nv = valid(at);
    float g = load_g(at, nv), through = 0.0f;
    bool ok = true, more = true, failed = false;
    uint32_t it = 0;
    for (; more; it++) {
        const uint32_t ph = it & 1;
        const int64_t t0 = at.chunk * C;
        const bool first = at.h == at.h_lo && at.pt == 0, last = at.h + 1 == at.h_hi && at.pt + 1 == ptiles;
        Place next = at;
        more = step(next);
        // decays: c_i and e^{c_i - (start of its run of 32)}
        {
            const float x[1] = {g};
            Two c[1];
            warp_cumsum<1>(x, c);
            if (half == 0) {
                s_head[tok] = ex2(c[0].h + c[0].l);
                s_c[tok] = c[0];  // within the run; completed below
                if (lane == 31) s_end[run] = c[0];
            }
        }
        const int nv_next = more ? valid(next) : 0;
        if (more) g = load_g(next, nv_next);
        ok = mbar_wait(&s_ld, ph);
        if (ok && tok >= nv && t0 + tok < a.L) {  // tokens beyond the row's length
            const uint32_t zero[16] = {};
            write_row(V, tok, half, zero);
            write_row(DY, tok, half, zero);
            if (first)
#pragma unroll
                for (int n = 0; n < NB; n++) {
                    write_row(Q + n * 16384, tok, half, zero);
                    write_row(K + n * 16384, tok, half, zero);
                }
        }
        if (tid == 0) bulk_wait_read();  // the last dv (dq, dk) has left its staging tile
        tc_fence_before();
        fence_proxy_async_smem();
        failed = __syncthreads_or(!ok);
        if (failed) break;
        if (tid == 0) {
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
        Two end[4];
        end[0] = s_end[0];
#pragma unroll
        for (int i = 1; i < 4; i++) end[i] = two_add(end[i - 1], s_end[i]);
        const Two before = run == 0 ? Two{0.0f, 0.0f} : (run == 1 ? end[0] : (run == 2 ? end[1] : end[2]));
        const Two mine = run == 0 ? end[0] : (run == 1 ? end[1] : (run == 2 ? end[2] : end[3]));
        const Two cj = two_add(before, s_c[tok]);
        const float up = a.scale * ex2(cj.h + cj.l), down = ex2(two_diff(end[3], cj)), tail = ex2(two_diff(mine, cj));
        uint32_t vr[16];
        {
            uint32_t x[16];
            read_row(DY, tok, half, x);
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const float2 f = mul2(unpack2<T>(x[i]), splat2(up));
                x[i] = pack2<T>(f.x, f.y);
            }
            write_row(DS, tok, half, x);
            read_row(V, tok, half, vr);
        }
        ok = mbar_wait(&s_m1, ph);
        tc_fence_after();
        {
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const float2 f = mul2(unpack2<T>(vr[i]), splat2(down));
                x[i] = pack2<T>(f.x, f.y);
            }
            write_row(V, tok, half, x);
        }
        // P, E and W by 32 x 32 blocks: row block `run`, column blocks 0 and 3 (half 0) or 1 and 2 (half 1)
        uint32_t pr[2][16];
        float col = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const int cb = k == 0 ? half : 3 - half;
            uint32_t er[16];
            if (cb >= run) {
                float s[32], d[32], wv[32];
                tmem_ld32(tS + my + 32 * cb, s);
                tmem_ld32(tD + my + 32 * cb, d);
                if (cb > run) {
                    const Two start = cb == 1 ? end[0] : (cb == 2 ? end[1] : end[2]);
                    const float2 f = splat2(tail * ex2(two_diff(start, mine)));
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 t = *reinterpret_cast<const float4*>(&s_head[32 * cb + j]);
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            const int i = j + 2 * u;
                            const float2 m = mul2(f, u == 0 ? make_float2(t.x, t.y) : make_float2(t.z, t.w));
                            const float2 sv = make_float2(s[i], s[i + 1]);
                            const float2 p = mul2(m, sv);
                            const float2 e = mul2(mul2(m, splat2(a.scale)), make_float2(d[i], d[i + 1]));
                            const float2 x = mul2(e, sv);
                            pr[k][i / 2] = pack2<T>(p.x, p.y);
                            er[i / 2] = pack2<T>(e.x, e.y);
                            wv[i] = x.x;
                            wv[i + 1] = x.y;
                        }
                    }
                } else {
                    const Two own = s_c[tok];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float4 c = *reinterpret_cast<const float4*>(&s_c[32 * cb + i]);
                        const float m0 = i >= lane ? ex2(two_diff({c.x, c.y}, own)) : 0.0f;
                        const float m1 = i + 1 >= lane ? ex2(two_diff({c.z, c.w}, own)) : 0.0f;
                        const float e0 = i >= lane ? a.scale * m0 * d[i] : 0.0f;
                        const float e1 = i + 1 >= lane ? a.scale * m1 * d[i + 1] : 0.0f;
                        pr[k][i / 2] = pack2<T>(i >= lane ? m0 * s[i] : 0.0f, i + 1 >= lane ? m1 * s[i + 1] : 0.0f);
                        er[i / 2] = pack2<T>(e0, e1);
                        wv[i] = i > lane ? e0 * s[i] : 0.0f;
                        wv[i + 1] = i + 1 > lane ? e1 * s[i + 1] : 0.0f;
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; i++) col += wv[i];
                s_row[run][32 * cb + lane] = column_sums(wv);
            } else {
#pragma unroll
                for (int i = 0; i < 16; i++) pr[k][i] = er[i] = 0;
            }
            // E: row j, columns 32 cb .. + 31 of two 64-column tiles
#pragma unroll
            for (int u = 0; u < 4; u++)
                *unit(E + (cb >> 1) * 16384, tok, (cb & 1) * 4 + u) = make_uint4(er[4 * u], er[4 * u + 1], er[4 * u + 2], er[4 * u + 3]);
        }
        tc_fence_before();
        __syncthreads();  // S and D have been read
        tc_fence_after();
        tmem_st16(tP + my + 16 * half, pr[0]);
        tmem_st16(tP + my + 16 * (3 - half), pr[1]);
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        ok = mbar_wait(&s_st, ph) && ok;
        failed = __syncthreads_or(!ok);
        if (failed) break;
        if (tid == 0) {
            tc_fence_after();
            constexpr uint32_t dV = mma_desc<T>(128, PT, false, true), dQ = mma_desc<T>(128, NP, true, true),
                               dQs = mma_desc<T>(128, NP, false, false), dK = mma_desc<T>(128, NP, false, true);
#pragma unroll
            for (int s = 0; s < C / 16; s++) mma_ts(tV, tP + 8 * s, smem_desc(smem_addr(DY) + s * 2048), dV, s > 0);
#pragma unroll
            for (int s = 0; s < 8 * NB; s++) {  // k R and q H, high and low parts
                const int n = s % (4 * NB);
                const uint32_t o = (n >> 2) * 16384 + (n & 3) * 32, st = (s / (4 * NB)) * NB * 8192 + n * 2048;
                mma(tF, smem_desc(smem_addr(K) + o), smem_desc(smem_addr(R) + st), dV, s > 0);
                mma(tZ, smem_desc(smem_addr(Q) + o), smem_desc(smem_addr(H) + st), dV, s > 0);
            }
            mma_commit(&s_m2);
#pragma unroll
            for (int s = 0; s < C / 16; s++) {
                mma(tQ, smem_desc(smem_addr(E) + s * 2048, 16384), smem_desc(smem_addr(K) + s * 2048, 16384), dQ, !first || s > 0);
                mma(tK, smem_desc(smem_addr(E) + (s >> 2) * 16384 + (s & 3) * 32), smem_desc(smem_addr(Q) + s * 2048, 16384), dK,
                    !first || s > 0);
            }
#pragma unroll
            for (int s = 0; s < PT / 16; s++) {
                mma(tQ, smem_desc(smem_addr(DS) + s * 32), smem_desc(smem_addr(H) + s * 32), dQs, true);
                mma(tK, smem_desc(smem_addr(V) + s * 32), smem_desc(smem_addr(R) + s * 32), dQs, true);
            }
            mma_commit(&s_m3);
        }
        // <R, H> of this tile: rows n of both, high + low
        if (at.pt == 0) through = 0.0f;
        if (tok < NP) {
            uint32_t h0[16], h1[16], r0[16], r1[16];
            read_row(H, tok, half, h0);
            read_row(H + NB * 8192, tok, half, h1);
            read_row(R, tok, half, r0);
            read_row(R + NB * 8192, tok, half, r1);
            float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 16; i++)
                acc = fma2(add2(unpack2<T>(h0[i]), unpack2<T>(h1[i])), add2(unpack2<T>(r0[i]), unpack2<T>(r1[i])), acc);
            through += acc.x + acc.y;
        }
        uint32_t dyr[16], dv[16];
        read_row(DY, tok, half, dyr);
        ok = mbar_wait(&s_m2, ph);
        tc_fence_after();
        {
            float f[32], x[32];
            tmem_ld32(tF + my + 32 * half, f);
            tmem_ld32(tV + my + 32 * half, x);
            float2 b = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const float2 y = mul2(splat2(down), make_float2(f[2 * i], f[2 * i + 1]));
                b = fma2(y, unpack2<T>(vr[i]), b);
                const float2 z = fma2(splat2(a.scale), make_float2(x[2 * i], x[2 * i + 1]), y);
                dv[i] = pack2<T>(z.x, z.y);
            }
            float sb = b.x + b.y + col;
            tmem_ld32(tZ + my + 32 * half, f);
            float2 z = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 16; i++) z = fma2(make_float2(f[2 * i], f[2 * i + 1]), unpack2<T>(dyr[i]), z);
            float sa = up * (z.x + z.y);
            if (half == 0)  // row_i, from the row blocks up to its own
                for (int r = 0; r <= run; r++) sb -= s_row[r][tok];
            if (at.pt > 0) {
                sa += s_a[half][tok];
                sb += s_b[half][tok];
            }
            s_a[half][tok] = sa;
            s_b[half][tok] = sb;
        }
        ok = mbar_wait(&s_m3, ph) && ok;
        tc_fence_after();
        write_row(DS, tok, half, dv);
        tc_fence_before();
        fence_proxy_async_smem();
        float th = through;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) th += __shfl_xor_sync(kFull, th, o);
        if (lane == 0) s_red[tid >> 5] = th;
        failed = __syncthreads_or(!ok);
        if (failed) break;
        if (tid == 0) {
            if (more) load(next);
            tma_store_4d(&w.maps.dv, DS, (int)(at.pt * PT), (int)at.h, (int)t0, (int)at.b);
            bulk_commit();
        }
        if (at.pt + 1 == ptiles && tid >= 224) {  // the last warp: dg of this head, tokens 4 lane .. 4 lane + 3
            float sum = 0.0f, av[4], bv[4];
#pragma unroll
            for (int u = 0; u < 8; u++) sum += s_red[u];
            sum *= ex2(end[3].h + end[3].l);
            float A = 0.0f, B = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                av[e] = s_a[0][4 * lane + e] + s_a[1][4 * lane + e];
                bv[e] = s_b[0][4 * lane + e] + s_b[1][4 * lane + e];
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
            float before_t = pre;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int t = 4 * lane + e;
                if (t0 + t < a.L) w.dg[(at.b * a.L + t0 + t) * a.H + at.h] = t < nv ? suf + before_t + sum : 0.0f;
                suf -= av[e];
                before_t += bv[e];
            }
        }
        if (last) {  // dq and dk of the group (or of this part of its heads)
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const uint32_t from = k == 0 ? tQ : tK;
                if (w.splits > 1) {
                    float* to = (k == 0 ? w.dq_part : w.dk_part) + at.split * a.Bsz * a.L * a.G * a.N +
                                ((at.b * a.L + t0 + tok) * a.G + at.gq) * a.N;
#pragma unroll
                    for (int c = 0; c < NB; c++) {
                        float x[32];
                        const int n0 = 32 * NB * half + 32 * c;
                        tmem_ld32(from + my + n0, x);
                        if (t0 + tok < a.L)
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                if (n0 + i < a.N)
                                    *reinterpret_cast<float4*>(to + n0 + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                    }
                } else {
                    // NB == 1: a tile of E for each; NB == 2: E for dq, then for dk
                    if (NB == 2 && k == 1) {
                        if (tid == 0) bulk_wait_read();
                        __syncthreads();
                    }
                    char* to = NB == 1 ? E + k * 16384 : E;
#pragma unroll
                    for (int c = 0; c < NB; c++) {
                        float x[32];
                        const int n0 = 32 * NB * half + 32 * c;
                        tmem_ld32(from + my + n0, x);
                        uint32_t r[16];
#pragma unroll
                        for (int i = 0; i < 16; i++) r[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
                        write_row(to + (n0 >> 6) * 16384, tok, (n0 >> 5) & 1, r);
                    }
                    fence_proxy_async_smem();
                    __syncthreads();
                    if (tid == 0) {
#pragma unroll
                        for (int n = 0; n < NB; n++)
                            tma_store_4d(k == 0 ? &w.maps.dq : &w.maps.dk, to + n * 16384, n * 64, (int)at.gq, (int)t0, (int)at.b);
                        bulk_commit();
                    }
                }
            }
        }
        at = next;
        nv = nv_next;
    }
    if (failed) {  // a wait ran out: report, wait for what is in flight (within limits), leave
        if (tid == 0) {
            atomicOr(w.status, kDevWaitTimeout);
            mbar_wait(&s_ld, it & 1);
            mbar_wait(&s_st, it & 1);
            mbar_wait(&s_m1, it & 1);
            mbar_wait(&s_m3, it & 1);
        }
    }
    if (tid == 0) bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (tid < 32) tmem_free(tm, 512);
}

template <typename T, int NB> cudaError_t bwd_n(const TcBwdArgs& w, cudaStream_t st) {
    constexpr int smem = BwdSmem<NB>::total;
    const cudaError_t e = cudaFuncSetAttribute(k_tc_bwd<T, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t items = w.a.Bsz * w.chunks * w.a.G * w.splits;
    k_tc_bwd<T, NB><<<(unsigned)(items < kSms ? items : kSms), 256, smem, st>>>(w);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tc_bwd(const TcBwdArgs& w, cudaStream_t st) {
    return w.a.N > 64 ? bwd_n<__nv_bfloat16, 2>(w, st) : bwd_n<__nv_bfloat16, 1>(w, st);
}

}  // namespace la
}  // namespace ss
