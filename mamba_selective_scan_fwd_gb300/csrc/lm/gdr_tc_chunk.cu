// Gated delta rule's backward on the tensor cores: one chunk of the heads that share a head
// of q and k, from the walks' images of H (state before the chunk), R (adjoint after it), U and X.
//
// Rows 0 .. 63 of every product belong to the tokens' keys, 64 .. 127 to their queries:
//   [K; Q] K^T                       kk, qk
//   [X; dY] U^T                      F = -beta e^{c_i - c_j} x_i . u_j (j < i),  E = scale e^{c_i - c_j} dy_i . u_j (j <= i)
//   [X; dY] H^T                      -beta e^c of it: k's share by H; scale e^c of it: q's
//   U R^T                            e^{cl - c} of it: k's share by R
//   [F; E] K,  [F; E]^T [K; Q]       the pairs' shares
// dq and dk stay in registers over the heads.  dv = beta x;  dbeta_i = x_i . v_i - e^{c_i} k_i . H x_i - sum_j e^{c_i - c_j}
// (k_i . k_j) (x_i . u_j);  dg is made of every path's two ends (gdr_f32.cu has the formula).
//
// An item's tiles fill shared memory, so one block an SM, and its products, the passes over their results and the loads of the
// next tiles wait for one another: 23 thousand cycles an item (28 of them in 333 us at 1.96 GHz), and the workers' registers
// spill some 500 bytes.  Blocks therefore stay on their SM and load the next unit's tiles under the last item's end.  2 x 4096
// tokens, 32 heads, N = P = 128, bf16: 346 us (with E and F in one part 310, and then a block a unit 350, tiles sent to the L2
// cache ahead 328 to 339).
//
// Roundings: H, R, U, X and the E and F of dq's and dk's products are f16 in two parts (22 bits), and dg and dbeta take all else
// in f32.  (E and F as one part are 10 % faster, but leave dq and dk of bf16 io 2^-12 off before their own rounding.)
#include "../simd.cuh"
#include "gdr_tc.cuh"

namespace ss {
namespace gdr {
namespace {

using la::pack2;
using la::Two;
using la::unit;
using la::unpack2;

constexpr int C = kChunk;
constexpr int kWorkers = 256, kThreads = kWorkers + 128;  // one thread of the last 128 loads and issues the products
// Registers a thread: 168 at launch; the workers take what the others leave (2 x 224 + 56 of 3 x 168).
__device__ __forceinline__ void take_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 224;"); }
__device__ __forceinline__ void leave_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;"); }

template <int NB> struct ChunkSmem {
    // K and Q by turns; X and dY (high parts); X's low part and zeros (dY has none); U, high and low; H or R, for each 64
    // states high and low; [F; E]
    static constexpr int keys = 0, z = NB * 16384, zl = z + 32768, u = zl + 32768, s = u + 32768, ef = s + NB * 32768, head = ef + 16384,
                         total = head + 2048;
};
constexpr uint32_t cE = 0, cQK = 64, cT = 0, cZ = 128, cR = 256, cK = 384;

__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void arrive(uint64_t* bar) {  // a warp's
    la::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) la::mbar_arrive(bar);
}
__device__ __forceinline__ float warp_max(float v) {
    uint32_t m;
    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(__float_as_uint(v)));
    return __uint_as_float(m);
}
template <int W> __device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
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
// eight f16 values . eight f32 values
__device__ __forceinline__ float dot8(uint4 k, const float* x, float sum) {
    const uint32_t v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float2 f = unpack2<__half>(v[e]);
        sum = fmaf(f.x, x[2 * e], fmaf(f.y, x[2 * e + 1], sum));
    }
    return sum;
}

// One chunk of (a part of) the heads that share a head of q and k.  An item is one of them, or 128 of its value channels.
struct Unit {
    int b, chunk, gq, split, h_lo, items, nv;
};

template <typename T, int NB> __global__ void __launch_bounds__(kThreads, 1) k_chunk(const __grid_constant__ TcChunkArgs w) {
    extern __shared__ __align__(1024) char sm[];
    using L = ChunkSmem<NB>;
    constexpr int W = 32 * NB;  // states of a thread
    // landed: K and Q; an item's tiles; H or R.  Workers: E and F stand; H is copied; the item's tiles are read, its products.
    // Products: E; H's; R's; the pairs'
    __shared__ __align__(8) uint64_t s_key, s_in, s_h[2], s_ef, s_copied, s_read, s_done, s_c1, s_c2, s_c3, s_c4;
    __shared__ uint32_t s_tm, s_fail;
    __shared__ float s_max[8], s_xv[4][C], s_row[2][128], s_col[8][32], s_dot[3][2][128], s_a[C], s_b[C], s_db[C], s_thr[8];
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = tid & 127, half = tid >> 7;
    const int ptiles = (int)((a.P + kTileP - 1) / kTileP);
    const uint32_t units = (uint32_t)(a.Bsz * w.chunks * a.G * w.splits);
    auto unit_of = [&](uint32_t id) {
        Unit u;
        const int rep = (int)a.H / (int)a.G;
        u.split = (int)(id % (uint32_t)w.splits);
        id /= (uint32_t)w.splits;
        u.gq = (int)(id % (uint32_t)a.G);
        id /= (uint32_t)a.G;
        u.chunk = (int)(id % (uint32_t)w.chunks);
        u.b = (int)(id / (uint32_t)w.chunks);
        u.h_lo = u.gq * rep + rep * u.split / w.splits;
        u.items = (u.gq * rep + rep * (u.split + 1) / w.splits - u.h_lo) * ptiles;
        u.nv = (int)max((int64_t)0, min((int64_t)C, row_length(a, u.b) - (int64_t)u.chunk * C));
        return u;
    };
    const bool q_side = r >= C;
    const int tok = r & (C - 1);
    const int n0 = half * W;  // this thread's states
    auto put_out = [&](const Unit& u, const float (&acc)[W]) {  // dq's or dk's row
        const int64_t t = (int64_t)u.chunk * C + tok;
        if (t >= a.L) return;
        const int64_t at = ((u.b * a.L + t) * a.G + u.gq) * a.N + n0;
        const bool on = tok < u.nv;
#pragma unroll
        for (int n = 0; n < W; n += 8) {
            if (n0 + n >= a.N) break;
            if (w.splits > 1) {
                float* to = (q_side ? w.dq_part : w.dk_part) + u.split * a.Bsz * a.L * a.G * a.N + at + n;
#pragma unroll
                for (int e = 0; e < 8; e += 4)
                    *reinterpret_cast<float4*>(to + e) = on ? make_float4(acc[n + e], acc[n + e + 1], acc[n + e + 2], acc[n + e + 3]) : make_float4(0, 0, 0, 0);
            } else {
                T* to = static_cast<T*>(q_side ? w.dq : w.dk) + at + n;
                uint32_t x[4];
#pragma unroll
                for (int e = 0; e < 4; e++) x[e] = on ? pack2<T>(acc[n + 2 * e], acc[n + 2 * e + 1]) : 0;
                *reinterpret_cast<uint4*>(to) = make_uint4(x[0], x[1], x[2], x[3]);
            }
        }
    };
    char *KQ = sm + L::keys, *Z = sm + L::z, *Zl = sm + L::zl, *U = sm + L::u, *S = sm + L::s, *EF = sm + L::ef;
    const ImageHead* head = reinterpret_cast<const ImageHead*>(sm + L::head);
    if (tid == 0) {
        for (uint64_t* bar : {&s_key, &s_in, &s_h[0], &s_h[1], &s_c1, &s_c2, &s_c3, &s_c4}) mbar_init(bar, 1);
        for (uint64_t* bar : {&s_ef, &s_copied, &s_read, &s_done}) mbar_init(bar, kWorkers / 32);
        s_fail = 0;
        fence_proxy_async_smem();
    }
    if (warp == 0) la::tmem_alloc(&s_tm, 512);
    for (int i = tid; i < kPieceBytes / 16; i += kThreads) *reinterpret_cast<uint4*>(Zl + kPieceBytes + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncthreads();
    la::tc_fence_after();
    const uint32_t tm = __shfl_sync(kFull, s_tm, 0), my = (uint32_t)(tid & 96) << 16;
    auto image_of = [&](const Unit& u, int item) { return ((u.b * a.H + u.h_lo + item / ptiles) * ptiles + item % ptiles) * w.chunks + u.chunk; };
    auto load_states = [&](const char* images, int64_t im, int n) {  // 64 of the states, two parts
        mbar_expect_tx(&s_h[n], 4 * kTileBytes);
#pragma unroll
        for (int part = 0; part < 2; part++)
            bulk_load(S + n * 32768 + part * 16384, images + im * state_bytes(NB) + (part * NB + n) * 16384, 16384, &s_h[n]);
    };
    auto load = [&](const Unit& u, int item) {
        const int64_t h = u.h_lo + item / ptiles, im = image_of(u, item);
        mbar_expect_tx(&s_in, 2 * kRowsBytes + kPieceBytes + (int)sizeof(ImageHead));
        bulk_load(sm + L::head, w.images + ((u.b * a.H + h) * w.chunks + u.chunk) * kImageBytes + 4 * kTileBytes, (int)sizeof(ImageHead), &s_in);
        bulk_load(Z, w.xs + im * kRowsBytes, kPieceBytes, &s_in);
        bulk_load(Zl, w.xs + im * kRowsBytes + kPieceBytes, kPieceBytes, &s_in);
        bulk_load(Z + kPieceBytes, w.dys + im * kPieceBytes, kPieceBytes, &s_in);
        bulk_load(U, w.us + im * kRowsBytes, kRowsBytes, &s_in);
        for (int n = 0; n < NB; n++) load_states(w.before, im, n);
    };
    if (warp >= kWorkers / 32) {
        leave_regs();
        if (__shfl_sync(kFull, warp, 0) == kWorkers / 32) {
            constexpr uint32_t kk = la::mma_desc<__half>(128, C, false, false), kw = la::mma_desc<__half>(128, 64 * NB, false, true),
                               rr = la::mma_desc<__half>(128, C, true, true), rw = la::mma_desc<__half>(128, 64 * NB, true, true);
            const uint32_t keys_at = smem_addr(KQ), z_at = smem_addr(Z), zl_at = smem_addr(Zl), u_at = smem_addr(U), s_at = smem_addr(S), ef_at = smem_addr(EF);
            auto load_keys = [&](const Unit& u) {
                mbar_expect_tx(&s_key, NB * 16384);
                bulk_load(KQ, w.keys + ((u.b * w.chunks + u.chunk) * a.G + u.gq) * (NB * 16384), NB * 16384, &s_key);
            };
            // units without a token are the workers' alone
            uint32_t id = blockIdx.x;
            Unit next;
            auto find = [&] {
                for (; id < units; id += gridDim.x) {
                    next = unit_of(id);
                    if (next.nv > 0) break;
                }
                id = __shfl_sync(kFull, id, 0);
            };
            find();
            uint32_t done = 0, keys = 0;
            if (lane == 0 && id < units) {
                load_keys(next);
                load(next, 0);
            }
            __syncwarp();
            bool ok = true;
            while (ok && id < units) {
                const Unit work = next;
                const int steps = __shfl_sync(kFull, work.items, 0);
                id += gridDim.x;
                find();
                ok = warp_wait(&s_key, keys++ & 1, &s_fail);
                for (int item = 0; item < steps; item++) {
                    const uint32_t ph = done++ & 1;
                    ok = false;
                    if (!warp_wait(&s_in, ph, &s_fail) || (done > 1 && !warp_wait(&s_done, ph ^ 1, &s_fail))) break;
                    la::tc_fence_after();
                    if (elect()) {
#pragma unroll
                        for (int s = 0; s < 4 * NB; s++) {
                            const uint32_t x = keys_at + (s >> 2) * 16384 + (s & 3) * 32;
                            la::mma(tm + cQK, la::smem_desc(x), la::smem_desc(x), kk, s > 0);
                        }
#pragma unroll
                        for (int o = 0; o < 3; o++)  // lo hi, hi lo, hi hi
#pragma unroll
                            for (int s = 0; s < 8; s++)
                                la::mma(tm + cE, la::smem_desc((o == 0 ? zl_at : z_at) + s * 2048, kPieceBytes), la::smem_desc(u_at + (o == 1 ? kPieceBytes : 0) + s * 2048), rr,
                                        o > 0 || s > 0);
                        la::mma_commit(&s_c1);
                    }
                    for (int n = 0; n < NB; n++) warp_wait(&s_h[n], 0, &s_fail);
                    // (all states at once: the left operand is read from shared memory half as often)
                    if (elect()) {
#pragma unroll
                        for (int o = 0; o < 3; o++)
#pragma unroll
                            for (int s = 0; s < 8; s++)
                                la::mma(tm + cZ, la::smem_desc((o == 0 ? zl_at : z_at) + s * 2048, kPieceBytes),
                                        la::smem_desc(s_at + (o == 1 ? kPieceBytes : 0) + s * 2048, 2 * kPieceBytes), rw, o > 0 || s > 0);
                        la::mma_commit(&s_c2);
                    }
                    // R takes H's place
                    if (!warp_wait(&s_copied, ph, &s_fail)) break;
                    warp_wait(&s_c2, ph, &s_fail);
                    if (lane == 0)
                        for (int n = 0; n < NB; n++) load_states(w.after, image_of(work, item), n);
                    __syncwarp();
                    if (!warp_wait(&s_ef, ph, &s_fail)) break;
                    la::tc_fence_after();
                    if (elect()) {
#pragma unroll
                        for (int part = 1; part >= 0; part--) {
                            const uint32_t left = part ? zl_at : ef_at;
#pragma unroll
                            for (int s = 0; s < 4; s++)
                                la::mma(tm + cK, la::smem_desc(left + s * 32), la::smem_desc(keys_at + s * 2048, 16384), kw, part < 1 || s > 0);
#pragma unroll
                            for (int s = 0; s < 8; s++)
                                la::mma(tm + cT, la::smem_desc(left + s * 2048, 0), la::smem_desc(keys_at + s * 2048, 16384), rw, part < 1 || s > 0);
                        }
                        la::mma_commit(&s_c4);
                    }
                    for (int n = 0; n < NB; n++) warp_wait(&s_h[n], 1, &s_fail);
                    // (the 64 tokens twice)
                    if (elect()) {
#pragma unroll
                        for (int o = 0; o < 3; o++)
#pragma unroll
                            for (int s = 0; s < 8; s++)
                                la::mma(tm + cR, la::smem_desc(u_at + (o == 0 ? kPieceBytes : 0) + s * 2048, 0),
                                        la::smem_desc(s_at + (o == 1 ? kPieceBytes : 0) + s * 2048, 2 * kPieceBytes), rw, o > 0 || s > 0);
                        la::mma_commit(&s_c3);
                    }
                    if (item + 1 < steps || id < units) {  // (E's and F's low part stands in Z's)
                        if (!warp_wait(&s_read, ph, &s_fail) || !warp_wait(&s_c3, ph, &s_fail) || !warp_wait(&s_c4, ph, &s_fail)) break;
                        if (lane == 0) {
                            if (item + 1 < steps) load(work, item + 1);
                            else load(next, 0);
                        }
                        __syncwarp();
                    }
                    ok = true;
                }
                if (ok && id < units) {  // the workers read K and Q to the item's end
                    ok = warp_wait(&s_done, (done & 1) ^ 1, &s_fail);
                    if (ok && lane == 0) load_keys(next);
                    __syncwarp();
                }
            }
        }
        __syncwarp();
    } else {
        take_regs();
        bool ok = true;
        uint32_t done = 0;  // items
        for (uint32_t id = blockIdx.x; id < units; id += gridDim.x) {
            const Unit work = unit_of(id);
            const int64_t b = work.b, t0 = (int64_t)work.chunk * C;
            const int nv = work.nv, nt = (int)min((int64_t)C, a.L - t0);
            float acc[W] = {};
            auto put_dv = [&](int64_t h, int64_t p0, int row, int u, uint4 x) {
                if (row < nt && p0 + 8 * u < a.P)
                    *reinterpret_cast<uint4*>(static_cast<T*>(w.dv) + ((b * a.L + t0 + row) * a.H + h) * a.P + p0 + 8 * u) = x;
            };
            if (nv == 0) {
                put_out(work, acc);
                for (int item = 0; item < work.items; item++) {
                    const int64_t h = work.h_lo + item / ptiles, p0 = (int64_t)(item % ptiles) * kTileP;
                    for (int i = tid; i < C * 16; i += kWorkers) put_dv(h, p0, i >> 4, i & 15, make_uint4(0, 0, 0, 0));
                    if (p0 == 0 && tid < nt) {
                        const int64_t at = (b * a.L + t0 + tid) * a.H + h;
                        if (w.dg) w.dg[at] = 0.0f;
                        w.dbeta[at] = 0.0f;
                    }
                }
                continue;
            }
            for (int item = 0; item < work.items; item++) {
                const uint32_t ph = done++ & 1;
                const int pt = item % ptiles;
                const int64_t h = work.h_lo + item / ptiles, p0 = (int64_t)pt * kTileP, im = image_of(work, item);
                const float x_inv = w.x_inv[im], dy_inv = w.dy_inv[im], u_inv = w.u_inv[im], before_inv = w.before_inv[im], after_inv = w.after_inv[im];
                if (pt == 0) {
                    if (tid >= 64 && tid < 64 + C) s_a[tid - 64] = s_b[tid - 64] = s_db[tid - 64] = 0.0f;
                    if (tid >= 128 && tid < 136) s_thr[tid - 128] = 0.0f;
                }
                // dv, and x . v: token tid & 63, a quarter of the channels
                const int vt = tid & (C - 1), vp = (tid >> 6) * 32;
                uint4 vv[4];
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    vv[u] = make_uint4(0, 0, 0, 0);
                    if (vt < nv && p0 + vp + 8 * u < a.P)
                        vv[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v.p) + b * a.v.batch + (t0 + vt) * a.v.token + h * a.P + p0 + vp + 8 * u);
                }
                ok = wait(&s_in, ph, &s_fail) && ok;
                // X and dY are in the adjoints' units, U in the values'
                auto rise = [&](int t) { return head->grown ? power2(head->rise[t]) : 1.0f; };
                {
                    const float beta = head->beta[vt] * rise(vt);
                    float sum = 0.0f;
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const uint32_t v[4] = {vv[u].x, vv[u].y, vv[u].z, vv[u].w};
                        uint32_t out[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            float f[2];
#pragma unroll
                            for (int i = 0; i < 2; i++) {
                                const int p = vp + 8 * u + 2 * e + i;
                                const int at = p * 128 + (((vt >> 3) ^ (p & 7)) << 4) + (vt & 7) * 2;
                                f[i] = x_inv * (__half2float(*reinterpret_cast<const __half*>(Z + at)) + __half2float(*reinterpret_cast<const __half*>(Zl + at)));
                            }
                            const float2 g = unpack2<T>(v[e]);
                            sum = fmaf(f[0], g.x, fmaf(f[1], g.y, sum));
                            out[e] = vt < nv ? pack2<T>(beta * f[0], beta * f[1]) : 0;
                        }
                        put_dv(h, p0, vt, vp / 8 + u, make_uint4(out[0], out[1], out[2], out[3]));
                    }
                    s_xv[tid >> 6][vt] = head->grown ? sum * rise(vt) / la::ldf(&head->grow[vt]) : sum;
                }
                // H's tiles go to registers, for <R, H>, and make room for R's
                uint4 hs[NB][8];
#pragma unroll
                for (int n = 0; n < NB; n++) {
                    ok = wait(&s_h[n], 0, &s_fail) && ok;
                    if (w.dg)
#pragma unroll
                        for (int i = 0; i < 8; i++) hs[n][i] = *reinterpret_cast<const uint4*>(S + n * 32768 + (tid + 256 * i) * 16);
                }
                arrive(&s_copied);
                ok = wait(&s_c1, ph, &s_fail) && ok;
                la::tc_fence_after();
                auto rate = [&](int t) { return head->grown ? head->beta[t] * la::ldf(&head->grow[t]) : head->beta[t]; };
                const float inv_k = head->inv_k, inv_q = head->inv_q, beta = rate(tok), rho = q_side ? inv_q / inv_k : 1.0f;
                float ef_scale;
                {
                    float e[32], k[32];
                    la::tmem_ld32(tm + my + cE + 32 * half, e);
                    la::tmem_ld32(tm + my + cQK + 32 * half, k);
                    const Two* c = reinterpret_cast<const Two*>(head->c);
                    const Two ci = c[tok];
                    const float f = rise(tok) * u_inv * (q_side ? a.scale * dy_inv : x_inv), kf = (q_side ? inv_q : inv_k) * inv_k;
                    const int last = q_side ? tok : tok - 1;
                    pair_factors(e, c, head->tail, head->flat != 0, 32 * half, ci, f, last);
                    // of a key's row: e^{c_i - c_j} x_i . u_j so far
                    float row = 0.0f, most = 0.0f;
                    const float sign = q_side ? 1.0f : -beta;
#pragma unroll
                    for (int j = 0; j < 32; j++) {
                        k[j] = 32 * half + j < tok ? kf * k[j] * e[j] : 0.0f;
                        row += k[j];
                        e[j] *= sign;
                        k[j] *= sign;
                        most = fmaxf(most, fabsf(e[j]));
                    }
                    s_row[half][r] = row;  // (without the sign: dbeta takes a key's as it is)
                    s_col[warp][lane] = column_sums(k);
                    most = warp_max(rho * most);
                    if (lane == 0) s_max[warp] = most;
                    workers_sync();
#pragma unroll
                    for (int i = 0; i < 8; i++) most = fmaxf(most, s_max[i]);
                    ef_scale = la::f16_scale(most) * rho;
                    ok = wait(&s_c2, ph, &s_fail) && ok;  // the low part takes Z's, which H's product is done with
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        uint32_t x[4], y[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            float2 f = mul2(splat2(ef_scale), make_float2(e[8 * u + 2 * i], e[8 * u + 2 * i + 1]));
                            x[i] = pack2<__half>(f.x, f.y);
                            f = fma2(unpack2<__half>(x[i]), splat2(-1.0f), f);
                            y[i] = pack2<__half>(f.x, f.y);
                        }
                        *unit(EF, r, 4 * half + u) = make_uint4(x[0], x[1], x[2], x[3]);
                        *unit(Zl, r, 4 * half + u) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                if (tid < C) {
                    const float rows_k = s_row[0][tid] + s_row[1][tid], rows_q = s_row[0][64 + tid] + s_row[1][64 + tid];
                    float col = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; i++) col += s_col[(tid >> 5) * 4 + i][tid & 31];
                    s_b[tid] += col - (rows_q - rate(tid) * rows_k);
                    s_db[tid] += ((s_xv[0][tid] + s_xv[1][tid]) + (s_xv[2][tid] + s_xv[3][tid])) - rows_k;
                }
                fence_proxy_async_smem();
                arrive(&s_ef);
                // H's products
                ok = wait(&s_c2, ph, &s_fail) && ok;
                la::tc_fence_after();
                const float up = head->up[tok] * rise(tok), down = head->down[tok], all = head->up[C - 1] * la::ldf(&head->grow[C - 1]);
                {
                    const float f = before_inv * (q_side ? a.scale * up * dy_inv : -beta * up * x_inv);
                    float dot = 0.0f;
#pragma unroll
                    for (int c = 0; c < NB; c++) {
                        float z[32];
                        la::tmem_ld32(tm + my + cZ + n0 + 32 * c, z);
#pragma unroll
                        for (int u = 0; u < 4; u++) dot = dot8(*unit(KQ + ((n0 + 32 * c) >> 6) * 16384, r, ((n0 + 32 * c) & 63) / 8 + u), z + 8 * u, dot);
#pragma unroll
                        for (int n = 0; n < 32; n++) acc[32 * c + n] = fmaf(f, z[n], acc[32 * c + n]);
                    }
                    s_dot[0][half][r] = (q_side ? inv_q * f : inv_k * f) * dot;                        // a
                    if (!q_side) s_dot[1][half][r] = -inv_k * before_inv * up * x_inv * dot;           // dbeta's share
                }
                if (w.dg) {
                    float through = 0.0f;
#pragma unroll
                    for (int n = 0; n < NB; n++) {
                        ok = wait(&s_h[n], 1, &s_fail) && ok;
                        // units tid + 256 i: the high part for i < 4, the low part of the same values 1024 units on
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const uint4 rh = *reinterpret_cast<const uint4*>(S + n * 32768 + (tid + 256 * i) * 16),
                                        rl = *reinterpret_cast<const uint4*>(S + n * 32768 + 16384 + (tid + 256 * i) * 16);
                            const uint32_t x[4] = {hs[n][i].x, hs[n][i].y, hs[n][i].z, hs[n][i].w}, y[4] = {hs[n][i + 4].x, hs[n][i + 4].y, hs[n][i + 4].z, hs[n][i + 4].w};
                            const uint32_t p[4] = {rh.x, rh.y, rh.z, rh.w}, q[4] = {rl.x, rl.y, rl.z, rl.w};
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const float2 f = add2(unpack2<__half>(x[e]), unpack2<__half>(y[e])), g = add2(unpack2<__half>(p[e]), unpack2<__half>(q[e]));
                                through = fmaf(f.x, g.x, fmaf(f.y, g.y, through));
                            }
                        }
                    }
                    through = lane_sum<32>(through);
                    if (lane == 0) s_thr[warp] += through * (before_inv * after_inv);
                }
                arrive(&s_read);  // (R's products are waited for where the next tiles are loaded)
                ok = wait(&s_c3, ph, &s_fail) && ok;
                ok = wait(&s_c4, ph, &s_fail) && ok;
                la::tc_fence_after();
                {
                    const float fk = inv_k / ef_scale, fr = down * u_inv * after_inv, ft = fk;  // (a key's row: rho is 1)
                    float dot = 0.0f;
#pragma unroll
                    for (int c = 0; c < NB; c++) {
                        float z[32];
                        la::tmem_ld32(tm + my + cK + n0 + 32 * c, z);
#pragma unroll
                        for (int n = 0; n < 32; n++) acc[32 * c + n] = fmaf(fk, z[n], acc[32 * c + n]);
                        la::tmem_ld32(tm + my + cR + n0 + 32 * c, z);
                        if (!q_side) {
#pragma unroll
                            for (int u = 0; u < 4; u++) dot = dot8(*unit(KQ + ((n0 + 32 * c) >> 6) * 16384, r, ((n0 + 32 * c) & 63) / 8 + u), z + 8 * u, dot);
#pragma unroll
                            for (int n = 0; n < 32; n++) acc[32 * c + n] = fmaf(fr, z[n], acc[32 * c + n]);
                        }
                        la::tmem_ld32(tm + my + cT + n0 + 32 * c, z);
                        if (!q_side)
#pragma unroll
                            for (int n = 0; n < 32; n++) acc[32 * c + n] = fmaf(ft, z[n], acc[32 * c + n]);
                    }
                    if (!q_side) s_dot[2][half][r] = inv_k * fr * dot;  // b
                }
                arrive(&s_done);
                workers_sync();
                if (tid < C) {
                    s_a[tid] += (s_dot[0][0][tid] + s_dot[0][1][tid]) + (s_dot[0][0][64 + tid] + s_dot[0][1][64 + tid]);
                    s_b[tid] += s_dot[2][0][tid] + s_dot[2][1][tid];
                    s_db[tid] += s_dot[1][0][tid] + s_dot[1][1][tid];
                }
                workers_sync();
                if (pt == ptiles - 1 && warp == 0) {
                    float sum = 0.0f;
#pragma unroll
                    for (int u = 0; u < 8; u++) sum += s_thr[u];
                    sum *= all;
                    const int t = 2 * lane;
                    const float a0 = s_a[t], a1 = s_a[t + 1], b0 = s_b[t], b1 = s_b[t + 1];
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
                            w.dbeta[at] = t + e < nv ? s_db[t + e] : 0.0f;
                        }
                }
                workers_sync();
            }
            if (ok) put_out(work, acc);
        }
    }
    uint64_t* const bars[8] = {&s_key, &s_in, &s_h[0], &s_h[1], &s_c1, &s_c2, &s_c3, &s_c4};
    la::end_block(&s_fail, w.status, bars, tm, 512);
}

template <typename T, int NB> cudaError_t chunks_go(const TcChunkArgs& c, cudaStream_t st) {
    constexpr int bytes = ChunkSmem<NB>::total;
    const cudaError_t e = la::allow_smem<k_chunk<T, NB>>(bytes);
    if (e != cudaSuccess) return e;
    const int64_t units = c.a.Bsz * c.chunks * c.a.G * c.splits;
    k_chunk<T, NB><<<(unsigned)(units < la::kSms ? units : la::kSms), kThreads, bytes, st>>>(c);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tc_chunks(const TcChunkArgs& c, cudaStream_t st) {
    if (c.a.dtype == 1) return c.a.N <= 64 ? chunks_go<__half, 1>(c, st) : chunks_go<__half, 2>(c, st);
    return c.a.N <= 64 ? chunks_go<__nv_bfloat16, 1>(c, st) : chunks_go<__nv_bfloat16, 2>(c, st);
}

}  // namespace gdr
}  // namespace ss
