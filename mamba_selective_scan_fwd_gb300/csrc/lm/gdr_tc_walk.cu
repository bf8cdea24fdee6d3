// Gated delta rule on the tensor cores: the walk over the chunks.
//
// One block walks the chunks of one segment of one (batch row, head, 128 value channels)
// with the state transposed: the value channels are the 128 lanes of tensor memory, so that
// a thread owns a channel (half of its N states, half of a chunk's tokens) and every
// left operand is written by the thread that will read the product's row:
//   D1 = S^T [K; Q]^T        [128 x 128]  S in two f16 parts, from tensor memory
//   X = beta (V^T - e^c D1)               two parts
//   D2 = X M^T = U^T         [128 x 2 x 64]  hi [hi; lo] + lo hi
//   D3 = (e^{cl - c} U)^T K  [128 x N]    two parts;  S <- e^{cl} S + D3, f32 in registers
//   y = scale (e^c S^T Q^T + U^T P^T)     off the chain: a third warpgroup writes it
// One thread copies a chunk's tiles one chunk ahead, one warp issues all products.  The chain of a
// chunk is three products and three passes through the registers, and bounds the walk: of some 7100 cycles
// (at 1.96 GHz) S's parts take 920, D1 1800, X 860, D2 800, U 1000, D3 980, the update 500 (the state's threads' clocks, of 6900
// then), the products themselves 2950.  One block fills an SM's registers, so that nothing runs in the gaps.
// 4 x 4096 tokens, 32 heads, N = P = 128, bf16: 242 us.  65536 tokens, 8 heads in 18 segments: 361 us for
// the sums, 235 for the walk.
//
// Every operand made here is f16 in two parts (22 bits) under a power of two per channel, taken from the channel's
// largest value, which its two threads exchange (for X by a bound instead: 245 us for 250, but a state of which a chunk leaves
// 2^-15 is off by 10^-4 of that), or for S and R from a bound of some 2^5 above it, which costs none of the 22 bits;
// the f32 state stays good to a few 1e-7.  P and U too, for either io type: with one part each a bf16 y would be rounded twice
// (2.6e-4 of itself off before its own 1.66e-3), for 1 to 3 % less time: 4 x 4096 tokens, 32 heads 383 us for 387, 65536 tokens,
// 8 heads 758 for 780.
#include "../simd.cuh"
#include "gdr_tc.cuh"

namespace ss {
namespace gdr {
namespace {

using la::pack2;
using la::unit;
using la::unpack2;

constexpr int C = kChunk;
constexpr int kStateThreads = 256, kThreads = 512;  // state; output; loads and products (one thread of the last 128)
// Registers a thread: 128 at launch; the state's threads take what the others leave (2 x 168 + 112 + 56 of 4 x 128, 120 for
// the threads that write y).
template <int N> __device__ __forceinline__ void take_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void leave_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// columns of tensor memory: S^T K^T, then parts of U; S^T Q^T (one product with it); X M^T in two halves, then D3; U^T P^T; parts of S;
// parts of X, then of e U
constexpr uint32_t kD1 = 0, kQ = 64, kD3 = 128, kY = 256, kS = 320, kX = 448;

// A stage of shared memory: tiles of K and Q by turns (not Q: kTcSum, kTcKeep), V, the image
template <int NB, bool Q> struct Stage {
    static constexpr int block = (Q ? 2 : 1) * kTileBytes;  // K (and Q) of 64 columns
    static constexpr int v = NB * block, image = v + 2 * kTileBytes, head = image + (Q ? 4 : 2) * kTileBytes,
                         bytes = head + 2048;
};

__device__ __forceinline__ void arrive(uint64_t* bar) {  // a warp's
    la::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) la::mbar_arrive(bar);
}
__device__ __forceinline__ void named_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// 32 columns at each of two places, one wait.
__device__ __forceinline__ void tmem_ld64(uint32_t a, float (&x)[32], uint32_t b, float (&y)[32]) {
    uint32_t r[32], q[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\ttcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15]), "=r"(q[16]), "=r"(q[17]), "=r"(q[18]), "=r"(q[19]), "=r"(q[20]), "=r"(q[21]), "=r"(q[22]), "=r"(q[23]), "=r"(q[24]), "=r"(q[25]), "=r"(q[26]), "=r"(q[27]), "=r"(q[28]), "=r"(q[29]), "=r"(q[30]), "=r"(q[31])
                 : "r"(a), "r"(b));
#pragma unroll
    for (int i = 0; i < 32; i++) {
        x[i] = __uint_as_float(r[i]);
        y[i] = __uint_as_float(q[i]);
    }
}

// 32 values times s as two f16 parts: 16 columns of tensor memory each
__device__ __forceinline__ void put2(uint32_t hi, uint32_t lo, const float* x, float s) {
    uint32_t r[16], q[16];
#pragma unroll
    for (int i = 0; i < 16; i++) {
        float2 f = mul2(make_float2(x[2 * i], x[2 * i + 1]), splat2(s));
        r[i] = pack2<__half>(f.x, f.y);
        f = fma2(unpack2<__half>(r[i]), splat2(-1.0f), f);
        q[i] = pack2<__half>(f.x, f.y);
    }
    la::tmem_st16(hi, r);
    la::tmem_st16(lo, q);
}
template <int N> __device__ __forceinline__ float max_abs(const float* x) {
    float m[4] = {};
#pragma unroll
    for (int i = 0; i < N; i += 4)
#pragma unroll
        for (int e = 0; e < 4; e++) m[e] = fmaxf(m[e], fabsf(x[i + e]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// The power of two for a row whose largest value is `most`; of a row of zeros it is the largest there is, so
// that it never decides a scale common to more rows.
__device__ __forceinline__ float scale_of(float most) { return most == 0.0f ? 8.507059173023462e37f : la::f16_scale(most); }
// (bounds of values near f32's largest pass it, the values do not)
__device__ __forceinline__ float finite(float bound) { return fminf(bound, 3.4028234e38f); }
__device__ __forceinline__ uint32_t hmul2(uint32_t x, uint32_t y) {
    const __half2 z = __hmul2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&z);
}
// Smallest of a warpgroup's positive values (all get it).  Two barriers.
__device__ __forceinline__ float group_min(float v, uint32_t* red, int id) {
    uint32_t m;
    asm volatile("redux.sync.min.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(__float_as_uint(v)));
    if ((threadIdx.x & 31) == 0) red[(threadIdx.x >> 5) & 3] = m;
    named_sync(id, 128);
    m = min(min(red[0], red[1]), min(red[2], red[3]));
    named_sync(id, 128);
    return __uint_as_float(m);
}

// The images' pieces leave through a ring of places in shared memory, one warpgroup writing a row of 128 bytes a
// thread: 32 columns of tensor memory (or registers) of pairs of f16, times a power of two.
constexpr int kRing = 3;
struct Ring {
    char* place;
    int next;
    __device__ __forceinline__ void put(const uint32_t (&x)[32], uint32_t f, char* to) {
        const int pl = threadIdx.x & 127;
        char* at = place + next * kPieceBytes;
        next = next + 1 == kRing ? 0 : next + 1;
        if (pl == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kRing - 1) : "memory");
        named_sync(5, 128);  // the place is free
#pragma unroll
        for (int u = 0; u < 8; u++) *unit(at, pl, u) = make_uint4(hmul2(x[4 * u], f), hmul2(x[4 * u + 1], f), hmul2(x[4 * u + 2], f), hmul2(x[4 * u + 3], f));
        fence_proxy_async_smem();
        named_sync(5, 128);
        if (pl == 0) {
            la::bulk_store(to, at, kPieceBytes);
            la::bulk_commit();
        }
    }
};
__device__ __forceinline__ void tmem_bits(uint32_t addr, uint32_t (&r)[32]) {
    float x[32];
    la::tmem_ld32(addr, x);
#pragma unroll
    for (int i = 0; i < 32; i++) r[i] = __float_as_uint(x[i]);
}

// blockIdx.y of kTcSum: 0 walks from zero (E), 1 from the identity without v (Phi).
template <typename T, int NB, TcWalkMode MODE> __device__ __forceinline__ void walk(const TcWalkArgs& w, char* sm) {
    constexpr bool SUM = MODE == kTcSum, OUT = MODE == kTcY, KEEP = MODE == kTcKeep;
    constexpr int W = 32 * NB;
    using L = Stage<NB, OUT>;
    // landed; stage free; S; D1; X; D2; e U; D3; U; U^T P^T; read by the third warpgroup: early, late
    __shared__ __align__(8) uint64_t s_full[2], s_free[2], s_s, s_d1, s_x, s_d2, s_u, s_d3, s_uy, s_y, s_early, s_late;
    __shared__ uint32_t s_tm, s_fail, s_red[4];
    __shared__ float s_most[2][128], s_ud[2][128], s_xm[2][128], s_um[2][128], s_ss[2][128], s_us[2][128];
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pl = tid & 127;
    const bool phi = SUM && blockIdx.y == 1;
    const int64_t width = phi ? a.N : a.P, ptiles = (a.P + kTileP - 1) / kTileP;
    int64_t id = blockIdx.x;
    const int64_t pt = id % ptiles, p0 = pt * kTileP;
    id /= ptiles;
    if (phi && pt > 0) return;  // N <= 128 columns
    const int64_t bh = id % (a.Bsz * a.H), seg = id / (a.Bsz * a.H);
    if (SUM && !phi && seg == w.plan.K - 1) return;  // nothing follows it
    const int64_t b = bh / a.H, h = bh % a.H, hq = h / (a.H / a.G);
    const int64_t len = row_length(a, b);
    const int64_t c_begin = seg * w.plan.seg, t_begin = c_begin * C, t_end = min(a.L, (c_begin + w.plan.seg) * C);
    const int chunks = (int)max((int64_t)0, (min(len, t_end) - t_begin + C - 1) / C);

    if (tid == 0) {
        for (uint64_t* bar : {&s_full[0], &s_full[1], &s_d1, &s_d2, &s_d3, &s_y}) mbar_init(bar, 1);
        for (uint64_t* bar : {&s_s, &s_x, &s_u, &s_uy}) mbar_init(bar, kStateThreads / 32);
        for (uint64_t* bar : {&s_early, &s_late}) mbar_init(bar, 4);
        for (uint64_t* bar : {&s_free[0], &s_free[1]}) mbar_init(bar, OUT ? 4 : kStateThreads / 32);
        s_fail = 0;
        fence_proxy_async_smem();
    }
    if (warp == 0) la::tmem_alloc(&s_tm, 512);
    __syncthreads();
    la::tc_fence_after();
    const uint32_t tm = __shfl_sync(kFull, s_tm, 0), my = (uint32_t)((warp & 3) * 32) << 16;
    char* staging = sm + 2 * L::bytes;
    auto valid = [&](int ch) { return (int)min((int64_t)C, len - (t_begin + (int64_t)ch * C)); };

    if (warp < kStateThreads / 32) {
        take_regs<168>();
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
        // X's and e U's scales are their own largest values, which the channel's two threads exchange: after strong decays
        // or corrections what is left of them is far below any bound.  S's comes from a bound that is known when the
        // update is done, by its largest value before.
        auto pair_sync = [&] { named_sync(1 + (warp & 3), 64); };
        auto max_over = [&](const float (&m)[2][128]) { return fmaxf(m[0][pl], m[1][pl]); };
        bool ok = true;
        // beta V of a chunk, and the largest value of the channel's, while S^T K^T is on its way
        float x[32];
        auto values = [&](int ch) {
            char* at = sm + (ch & 1) * L::bytes;
            const ImageHead* head = reinterpret_cast<const ImageHead*>(at + L::head);
            ok = ok && wait(&s_full[ch & 1], (ch >> 1) & 1, &s_fail);
            if (phi) {
#pragma unroll
                for (int j = 0; j < 32; j++) x[j] = 0.0f;
            } else {
                const char* tile = at + L::v + (pl >> 6) * kTileBytes + (pl & 7) * 2;
                const int c = (pl & 63) >> 3;
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 be = *reinterpret_cast<const float4*>(&head->beta[32 * half + j]);
                    const float bs[4] = {be.x, be.y, be.z, be.w};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int t = 32 * half + j + e;
                        x[j + e] = bs[e] * ldf(reinterpret_cast<const T*>(tile + t * 128 + ((c ^ (t & 7)) << 4)));
                    }
                }
                const int nv = valid(ch);
                if (nv < C) {
#pragma unroll
                    for (int j = 0; j < 32; j++)
                        if (32 * half + j >= nv) x[j] = 0.0f;
                }
            }
        };
        s_most[half][pl] = max_abs<W>(S);
        pair_sync();
        float bound = max_over(s_most);  // of |S|
        pair_sync();
        for (int ch = 0; ch < chunks; ch++) {
            const uint32_t ph = ch & 1;
            char* at = sm + ph * L::bytes;
            const ImageHead* head = reinterpret_cast<const ImageHead*>(at + L::head);
            const int nv = valid(ch);
            const float ss = scale_of(bound);
            if (KEEP && ch > 0) ok = ok && wait(&s_early, ph ^ 1, &s_fail);  // the last parts have been copied
            if (!SUM && half == 0) s_ss[ph][pl] = ss;
#pragma unroll
            for (int c = 0; c < NB; c++) {
                const uint32_t to = tm + my + kS + half * (W / 2) + 16 * c;
                put2(to, to + 32 * NB, S + 32 * c, ss);
            }
            la::tmem_wait_st();
            arrive(&s_s);
            values(ch);
            const float inv1 = -head->inv_k / ss, k_most = head->most_k;
            ok = ok && wait(&s_d1, ph, &s_fail);
            la::tc_fence_after();
            float d[32];
            la::tmem_ld32(tm + my + kD1 + 32 * half, d);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&head->beta_up[32 * half + j]);
                const float2 y = fma2(mul2(splat2(inv1), make_float2(f.x, f.y)), make_float2(d[j], d[j + 1]), make_float2(x[j], x[j + 1]));
                const float2 z = fma2(mul2(splat2(inv1), make_float2(f.z, f.w)), make_float2(d[j + 2], d[j + 3]), make_float2(x[j + 2], x[j + 3]));
                x[j] = y.x;
                x[j + 1] = y.y;
                x[j + 2] = z.x;
                x[j + 3] = z.y;
            }
            if (nv < C) {  // (whatever S^T k is there)
#pragma unroll
                for (int j = 0; j < 32; j++)
                    if (32 * half + j >= nv) x[j] = 0.0f;
            }
            s_xm[half][pl] = max_abs<32>(x);
            pair_sync();
            const float x_most = max_over(s_xm), xs = scale_of(x_most);
            {
                const uint32_t to = tm + my + kX + 16 * half;
                put2(to, to + 32, x, xs);
            }
            la::tmem_wait_st();
            arrive(&s_x);
            const float inv2 = head->inv_m / xs;
            s_most[half][pl] = max_abs<W>(S);
            ok = ok && wait(&s_d2, ph, &s_fail);
            la::tc_fence_after();
            tmem_ld64(tm + my + kD3 + 64 + 32 * half, x, tm + my + kD3 + 32 * half, d);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const float2 f = mul2(splat2(inv2), add2(make_float2(d[j], d[j + 1]), make_float2(x[j], x[j + 1])));
                x[j] = f.x;
                x[j + 1] = f.y;
            }
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&head->down[32 * half + j]);
                const float2 y = mul2(make_float2(x[j], x[j + 1]), make_float2(f.x, f.y)), z = mul2(make_float2(x[j + 2], x[j + 3]), make_float2(f.z, f.w));
                d[j] = y.x;
                d[j + 1] = y.y;
                d[j + 2] = z.x;
                d[j + 3] = z.y;
            }
            s_ud[half][pl] = max_abs<32>(d);
            pair_sync();
            const float ud_most = max_over(s_ud), us = scale_of(ud_most);
            {
                const uint32_t to = tm + my + kX + 16 * half;
                put2(to, to + 32, d, us);
            }
            la::tmem_wait_st();
            const float by = head->by, keep = head->weak ? 1.0f : 0.0f, inv3 = head->inv_k / us;
            bound = finite(fmaf(64.0f * k_most, ud_most, max_over(s_most) * (keep + fabsf(by))));
            arrive(&s_u);
            if (!SUM) {
                // U's image is what the backward sums products of: its own largest value, off the chain.  For y a bound
                // does: parts of f16 keep 22 bits of rows that are 2^14 below theirs.
                float most = finite(64.0f * head->most_m * x_most);
                if (KEEP) {
                    s_um[half][pl] = max_abs<32>(x);
                    pair_sync();
                    most = max_over(s_um);
                }
                const float uy = scale_of(most);
                if (half == 0) s_us[ph][pl] = uy;
                const uint32_t to = tm + my + kD1 + 16 * half;
                put2(to, to + 32, x, uy);
                la::tmem_wait_st();
                arrive(&s_uy);
            }
            ok = ok && wait(&s_d3, ph, &s_fail);
            la::tc_fence_after();
            if (!OUT) arrive(&s_free[ph]);
#pragma unroll
            for (int c = 0; c < NB; c++) {
                la::tmem_ld32(tm + my + kD3 + half * W + 32 * c, d);
#pragma unroll
                for (int n = 0; n < 32; n += 2) {
                    const float2 o = make_float2(S[32 * c + n], S[32 * c + n + 1]);
                    // S + (e^cl - 1) S for a weak decay, e^cl S else (la::Decay)
                    const float2 f = fma2(splat2(inv3), make_float2(d[n], d[n + 1]), fma2(splat2(by), o, mul2(splat2(keep), o)));
                    S[32 * c + n] = f.x;
                    S[32 * c + n + 1] = f.y;
                }
            }
        }
        if (mine && ok) {
            float* to = nullptr;
            if (phi) {  // transposed: column p in a row
                float* col = w.seg_phi + (bh * w.plan.K + seg) * a.N * a.N + p * a.N;
#pragma unroll
                for (int n = 0; n < W; n += 4)
                    if (half * W + n < a.N) *reinterpret_cast<float4*>(col + half * W + n) = make_float4(S[n], S[n + 1], S[n + 2], S[n + 3]);
                if (w.seg_phi_t) to = w.seg_phi_t + (bh * w.plan.K + seg) * a.N * a.N;
            } else if (SUM) to = w.seg_state + (bh * w.plan.K + seg) * a.N * a.P;
            else if (seg == w.plan.K - 1 && w.last) to = w.last + bh * a.N * a.P;
            if (to)
#pragma unroll
                for (int n = 0; n < W; n++)
                    if (half * W + n < a.N) to[(half * W + n) * width + p] = S[n];
        }
    } else if (warp < kStateThreads / 32 + 4) {
        leave_regs<OUT ? 120 : 112>();
        const bool first = tid == kStateThreads;
        if (OUT) {
            T* yp = static_cast<T*>(w.yp) + (b * a.L * a.H + h) * a.P;
            const bool wide = p0 + 64 < a.P;
            for (int ch = 0; ch < chunks; ch++) {
                const uint32_t ph = ch & 1;
                const ImageHead* head = reinterpret_cast<const ImageHead*>(sm + ph * L::bytes + L::head);
                const int nv = valid(ch);
                wait(&s_full[ph], (ch >> 1) & 1, &s_fail);
                wait(&s_d1, ph, &s_fail);
                la::tc_fence_after();
                float2 q[32];
                {
                    const float2 inv = splat2(a.scale * head->inv_q / s_ss[ph][pl]);
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        float x[32];
                        la::tmem_ld32(tm + my + kQ + 32 * hf, x);
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            q[16 * hf + j / 2] = mul2(mul2(inv, *reinterpret_cast<const float2*>(&head->up[32 * hf + j])), make_float2(x[j], x[j + 1]));
                    }
                }
                arrive(&s_early);
                if (first) la::bulk_wait_read();
                named_sync(5, 128);  // the staging tiles are free
                wait(&s_y, ph, &s_fail);
                la::tc_fence_after();
                const float2 inv = splat2(a.scale * head->inv_p / s_us[ph][pl]);
                char* tile = staging + (pl >> 6) * kTileBytes + (pl & 7) * 2;
                const int cu = (pl & 63) >> 3;
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    float y[32];
                    la::tmem_ld32(tm + my + kY + 32 * hf, y);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const int t = 32 * hf + j;
                        const float2 x = mul2(fma2(inv, make_float2(y[j], y[j + 1]), q[t / 2]), unpack2<__nv_bfloat16>(*reinterpret_cast<const uint32_t*>(&head->grow[t])));
                        st(reinterpret_cast<T*>(tile + t * 128 + ((cu ^ (t & 7)) << 4)), t < nv ? x.x : 0.0f);
                        st(reinterpret_cast<T*>(tile + (t + 1) * 128 + ((cu ^ ((t + 1) & 7)) << 4)), t + 1 < nv ? x.y : 0.0f);
                    }
                }
                arrive(&s_late);
                arrive(&s_free[ph]);
                fence_proxy_async_smem();
                named_sync(5, 128);
                if (first) {
                    const int64_t t0 = t_begin + (int64_t)ch * C;
                    la::tma_store_4d(&w.y, staging, (int)p0, (int)h, (int)t0, (int)b);
                    if (wide) la::tma_store_4d(&w.y, staging + kTileBytes, (int)p0 + 64, (int)h, (int)t0, (int)b);
                    la::bulk_commit();
                }
            }
            // tokens of chunks beyond the row's length
            for (int64_t t = t_begin + (int64_t)chunks * C + (warp & 3); t < t_end; t += 4)
                for (int64_t p = p0 + lane * 8; p < min(a.P, p0 + kTileP); p += 256)
                    *reinterpret_cast<uint4*>(yp + t * a.H * a.P + p) = make_uint4(0, 0, 0, 0);
        }
        if (KEEP) {
            Ring ring = {staging, 0};
            for (int ch = 0; ch < chunks; ch++) {
                const uint32_t ph = ch & 1;
                const int64_t image = (bh * ptiles + pt) * w.chunks + c_begin + ch;
                uint32_t x[32];
                wait(&s_s, ph, &s_fail);
                la::tc_fence_after();
                // the parts of S under one scale: what the largest channel's is
                float own = s_ss[ph][pl], all = group_min(own, s_red, 5);
                uint32_t f = pack2<__half>(all / own, all / own);
                if (first) w.state_inv[image] = 1.0f / all;
#pragma unroll 1
                for (int c = 0; c < 2 * NB; c++) {
                    tmem_bits(tm + my + kS + 32 * c, x);
                    if (c == 2 * NB - 1) arrive(&s_early);
                    ring.put(x, f, w.states + image * state_bytes(NB) + c * kPieceBytes);
                }
                wait(&s_uy, ph, &s_fail);
                la::tc_fence_after();
                own = s_us[ph][pl], all = group_min(own, s_red, 5);
                f = pack2<__half>(all / own, all / own);
                if (first) w.u_inv[image] = 1.0f / all;
#pragma unroll 1
                for (int part = 0; part < 2; part++) {
                    tmem_bits(tm + my + kD1 + 32 * part, x);
                    if (part == 1) arrive(&s_late);
                    ring.put(x, f, w.us + image * kRowsBytes + part * kPieceBytes);
                }
            }
        }
        if (first) la::bulk_wait_all();
    } else {
        leave_regs<56>();
        const int role = __shfl_sync(kFull, warp, 0) - (kThreads - 128) / 32, steps = __shfl_sync(kFull, chunks, 0);
        if (role == 1 && lane == 0) {  // loads
            const char* keys = w.keys + ((b * w.chunks + c_begin) * a.G + hq) * (NB * 2 * kTileBytes);
            const char* images = w.images + (bh * w.chunks + c_begin) * kImageBytes;
            auto load = [&](int ch) {
                char* at = sm + (ch & 1) * L::bytes;
                uint64_t* bar = &s_full[ch & 1];
                const int t0 = (int)(t_begin + (int64_t)ch * C);
                mbar_expect_tx(bar, (OUT ? 2 : 1) * NB * kTileBytes + (phi ? 0 : 2 * kTileBytes) + (OUT ? 4 : 2) * kTileBytes +
                                        (int)sizeof(ImageHead));
                const char* kq = keys + ch * a.G * (NB * 2 * kTileBytes);
#pragma unroll
                for (int n = 0; n < NB; n++) bulk_load(at + n * L::block, kq + n * 2 * kTileBytes, L::block, bar);
                if (!phi) {
                    la::tma_load_4d(at + L::v, &w.v, (int)p0, (int)h, t0, (int)b, bar);
                    la::tma_load_4d(at + L::v + kTileBytes, &w.v, (int)p0 + 64, (int)h, t0, (int)b, bar);
                }
                const char* im = images + (int64_t)ch * kImageBytes;
                bulk_load(at + L::image, im, (OUT ? 4 : 2) * kTileBytes, bar);
                bulk_load(at + L::head, im + 4 * kTileBytes, (int)sizeof(ImageHead), bar);
            };
            for (int ch = 0; ch < chunks; ch++) {
                if (ch > 1 && !wait(&s_free[ch & 1], ((ch >> 1) + 1) & 1, &s_fail)) break;
                load(ch);
            }
        } else if (role == 0) {  // products
            // (A product of 16 terms takes 94 cycles with 128 columns of the right operand, 79 with 64.  Handing the high parts
            // over before the low ones are made: 248 -> 244 us on 4 x 4096 tokens, 32 heads, but the backward's walks 270 -> 283,
            // since stores and products share tensor memory.)
            for (int ch = 0; ch < steps; ch++) {
                const uint32_t ph = ch & 1;
                const uint32_t at = smem_addr(sm + ph * L::bytes), M = at + L::image, P = M + 2 * kTileBytes;
                constexpr uint32_t d1 = la::mma_desc<__half>(128, OUT ? 2 * C : C, false, false), d2 = la::mma_desc<__half>(128, 2 * C, false, false),
                                   dP = la::mma_desc<__half>(128, C, false, false), d3 = la::mma_desc<__half>(128, 64 * NB, false, true);
                if (!warp_wait(&s_full[ph], (ch >> 1) & 1, &s_fail)) break;
                // U of the chunk before has left its columns, and so has Q's product
                if (!SUM && ch > 0 && !warp_wait(OUT ? &s_y : &s_late, ph ^ 1, &s_fail)) break;
                if (OUT && ch > 0 && !warp_wait(&s_early, ph ^ 1, &s_fail)) break;
                if (!warp_wait(&s_s, ph, &s_fail)) break;
                la::tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int part = 1; part >= 0; part--)
#pragma unroll
                        for (int s = 0; s < 4 * NB; s++)
                            la::mma_ts(tm + kD1, tm + kS + part * 32 * NB + 8 * s, la::smem_desc(at + (s >> 2) * L::block + (s & 3) * 32), d1, part < 1 || s > 0);
                    la::mma_commit(&s_d1);
                }
                if (!warp_wait(&s_x, ph, &s_fail)) break;
                la::tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int s = 0; s < 4; s++) la::mma_ts(tm + kD3, tm + kX + 8 * s, la::smem_desc(M + s * 32), d2, s > 0);  // hi [hi; lo]
#pragma unroll
                    for (int s = 0; s < 4; s++) la::mma_ts(tm + kD3 + 64, tm + kX + 32 + 8 * s, la::smem_desc(M + s * 32), dP, true);  // lo hi
                    la::mma_commit(&s_d2);
                }
                if (!warp_wait(&s_u, ph, &s_fail)) break;
                la::tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int part = 1; part >= 0; part--)
#pragma unroll
                        for (int s = 0; s < 4; s++)
                            la::mma_ts(tm + kD3, tm + kX + part * 32 + 8 * s, la::smem_desc(at + s * 2048, L::block), d3, part < 1 || s > 0);
                    la::mma_commit(&s_d3);
                }
                if (OUT) {
                    if (!warp_wait(&s_uy, ph, &s_fail) || (ch > 0 && !warp_wait(&s_late, ph ^ 1, &s_fail))) break;
                    la::tc_fence_after();
                    if (elect()) {
#pragma unroll
                        for (int o = 0; o < 3; o++)  // lo hi, hi lo, hi hi
#pragma unroll
                            for (int s = 0; s < 4; s++)
                                la::mma_ts(tm + kY, tm + kD1 + (o == 0 ? 32 : 0) + 8 * s, la::smem_desc(P + (o == 1 ? kTileBytes : 0) + s * 32), dP,
                                           o > 0 || s > 0);
                        la::mma_commit(&s_y);
                    }
                }
            }
        }
    }
    __syncwarp();
    uint64_t* const bars[6] = {&s_full[0], &s_full[1], &s_d1, &s_d2, &s_d3, &s_y};
    la::end_block(&s_fail, w.status, bars, tm, 512);
}

template <typename T, int NB, TcWalkMode MODE>
__global__ void __launch_bounds__(kThreads, 1) k_walk(const __grid_constant__ TcWalkArgs w) {
    extern __shared__ __align__(1024) char sm[];
    walk<T, NB, MODE>(w, sm);
}

// ---------------------------------------------------------------- the backward's walk
// From the last chunk, with R the adjoint of the state after the chunk, transposed like S:
//   D0 = dY^T P              D1 = R^T K^T          dU = scale D0 + e^{cl - c} D1      (the adjoint of U)
//   D2 = dU M = X^T          (the adjoint of beta (v - ..), transposed)
//   Dq = (scale e^c dY)^T Q  D3 = (-beta e^c X)^T K     R <- e^{cl} R + Dq + D3
// D0 and Dq do not wait for R.  D0's left operand is dY's image, exact; the third warpgroup makes Dq's, and copies the
// parts of R and X that the chunk kernel reads.
template <int NB> struct BackStage {
    static constexpr int block = 2 * kTileBytes, dy = NB * block, image = dy + 2 * kTileBytes, head = image + 4 * kTileBytes,
                         bytes = head + 2048;
};
// columns: D1, then parts of X; D0, then D2; Dq, then D3; parts of R; parts of dU, then of -beta e^c X; parts of
// scale e^c dY
constexpr uint32_t bD1 = 0, bD0 = 64, bD3 = 128, bR = 256, bX = 384, bDq = 448;

// SUM: a segment's, from an adjoint of zero; no images.
template <int NB, bool SUM> __device__ __forceinline__ void walk_back(const TcWalkArgs& w, const TcBackArgs& r, int64_t id, char* sm) {
    constexpr int W = 32 * NB;
    using L = BackStage<NB>;
    __shared__ __align__(8) uint64_t s_full[2], s_free[2], s_r, s_d1, s_dq, s_x, s_d2, s_u, s_d3, s_dyq, s_xi, s_early, s_late;
    __shared__ uint32_t s_tm, s_fail, s_red[4];
    __shared__ float s_most[2][128], s_ud[2][128], s_xe[2][128], s_xm[2][128], s_rs[2][128], s_xsc[2][128], s_dqs[2][128];
    const Args& a = w.a;
    const int tid = threadIdx.x, warp = tid >> 5, pl = tid & 127;
    const int64_t ptiles = (a.P + kTileP - 1) / kTileP, pt = id % ptiles, p0 = pt * kTileP, bh = id / ptiles % (a.Bsz * a.H), seg = id / ptiles / (a.Bsz * a.H);
    const int64_t b = bh / a.H, h = bh % a.H, hq = h / (a.H / a.G), len = row_length(a, b), c_begin = seg * w.plan.seg;
    if (SUM && seg == 0) return;  // nothing comes before it
    const int chunks = (int)max((int64_t)0, min((len + C - 1) / C, c_begin + w.plan.seg) - c_begin);
    if (tid == 0) {
        for (uint64_t* bar : {&s_full[0], &s_full[1], &s_d1, &s_dq, &s_d2, &s_d3}) mbar_init(bar, 1);
        for (uint64_t* bar : {&s_r, &s_x, &s_u, &s_xi}) mbar_init(bar, kStateThreads / 32);
        for (uint64_t* bar : {&s_dyq, &s_early, &s_late}) mbar_init(bar, 4);
        for (uint64_t* bar : {&s_free[0], &s_free[1]}) mbar_init(bar, kStateThreads / 32 + 4);
        s_fail = 0;
        fence_proxy_async_smem();
    }
    if (warp == 0) la::tmem_alloc(&s_tm, 512);
    __syncthreads();
    la::tc_fence_after();
    const uint32_t tm = __shfl_sync(kFull, s_tm, 0), my = (uint32_t)((warp & 3) * 32) << 16;
    char* staging = sm + 2 * L::bytes;
    auto chunk_of = [&](int i) { return (int)c_begin + chunks - 1 - i; };
    const int64_t images = (bh * ptiles + pt) * w.chunks;

    if (warp < kStateThreads / 32) {
        take_regs<168>();
        const int half = tid >> 7;
        const int64_t p = p0 + pl;
        const bool mine = p < a.P;
        float R[W];
        float* const seg_state = w.plan.K > 1 ? r.seg_state + (bh * w.plan.K + seg) * a.N * a.P : nullptr;
        const float* from = SUM ? nullptr : seg_state ? seg_state : r.init ? r.init + bh * a.N * a.P : nullptr;
#pragma unroll
        for (int n = 0; n < W; n++) R[n] = from && mine && half * W + n < a.N ? from[(half * W + n) * a.P + p] : 0.0f;
        auto pair_sync = [&] { named_sync(1 + (warp & 3), 64); };
        auto max_over = [&](const float (&m)[2][128]) { return fmaxf(m[0][pl], m[1][pl]); };
        bool ok = true;
        s_most[half][pl] = max_abs<W>(R);
        pair_sync();
        float bound = max_over(s_most);
        pair_sync();
        for (int i = 0; i < chunks; i++) {
            const uint32_t ph = i & 1;
            char* at = sm + ph * L::bytes;
            const ImageHead* head = reinterpret_cast<const ImageHead*>(at + L::head);
            const float rs = scale_of(bound), dy_inv = r.dy_inv[images + chunk_of(i)];
            if (!SUM && i > 0) ok = ok && wait(&s_early, ph ^ 1, &s_fail);
            if (half == 0) s_rs[ph][pl] = rs;
#pragma unroll
            for (int c = 0; c < NB; c++) {
                const uint32_t to = tm + my + bR + half * (W / 2) + 16 * c;
                put2(to, to + 32 * NB, R + 32 * c, rs);
            }
            la::tmem_wait_st();
            arrive(&s_r);
            s_most[half][pl] = max_abs<W>(R);
            pair_sync();
            const float r_most = max_over(s_most);
            ok = ok && wait(&s_full[ph], (i >> 1) & 1, &s_fail);
            const float k_most = head->most_k, inv1 = head->inv_k / rs;
            ok = ok && wait(&s_d1, ph, &s_fail);  // D0 and D1
            la::tc_fence_after();
            const float inv0 = a.scale * head->inv_p * dy_inv;
            float x[32], d[32];
            tmem_ld64(tm + my + bD1 + 32 * half, x, tm + my + bD0 + 32 * half, d);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&head->down[32 * half + j]);
                const float2 y = fma2(mul2(splat2(inv1), make_float2(f.x, f.y)), make_float2(x[j], x[j + 1]), mul2(splat2(inv0), make_float2(d[j], d[j + 1])));
                const float2 z = fma2(mul2(splat2(inv1), make_float2(f.z, f.w)), make_float2(x[j + 2], x[j + 3]), mul2(splat2(inv0), make_float2(d[j + 2], d[j + 3])));
                x[j] = y.x;
                x[j + 1] = y.y;
                x[j + 2] = z.x;
                x[j + 3] = z.y;
            }
            s_xe[half][pl] = max_abs<32>(x);
            pair_sync();
            const float xs = scale_of(max_over(s_xe));
            {
                const uint32_t to = tm + my + bX + 16 * half;
                put2(to, to + 32, x, xs);
            }
            la::tmem_wait_st();
            arrive(&s_x);
            // Dq, while D2 is on its way
            ok = ok && wait(&s_dq, ph, &s_fail);
            la::tc_fence_after();
            const float by = head->by, keep = head->weak ? 1.0f : 0.0f, dqs = s_dqs[ph][pl], invq = head->inv_q / dqs;
#pragma unroll
            for (int c = 0; c < NB; c++) {
                la::tmem_ld32(tm + my + bD3 + half * W + 32 * c, d);
#pragma unroll
                for (int n = 0; n < 32; n += 2) {
                    const float2 o = make_float2(R[32 * c + n], R[32 * c + n + 1]);
                    const float2 f = fma2(splat2(invq), make_float2(d[n], d[n + 1]), fma2(splat2(by), o, mul2(splat2(keep), o)));
                    R[32 * c + n] = f.x;
                    R[32 * c + n + 1] = f.y;
                }
            }
            const float inv2 = head->inv_m / xs;
            ok = ok && wait(&s_d2, ph, &s_fail);
            la::tc_fence_after();
            la::tmem_ld32(tm + my + bD0 + 32 * half, x);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&head->beta_up[32 * half + j]);
                const float2 y = mul2(splat2(inv2), make_float2(x[j], x[j + 1])), z = mul2(splat2(inv2), make_float2(x[j + 2], x[j + 3]));
                x[j] = y.x;
                x[j + 1] = y.y;
                x[j + 2] = z.x;
                x[j + 3] = z.y;
                d[j] = -f.x * y.x;
                d[j + 1] = -f.y * y.y;
                d[j + 2] = -f.z * z.x;
                d[j + 3] = -f.w * z.y;
            }
            s_ud[half][pl] = max_abs<32>(d);
            pair_sync();
            const float ud_most = max_over(s_ud), us = scale_of(ud_most), inv3 = head->inv_k / us;
            {
                const uint32_t to = tm + my + bX + 16 * half;
                put2(to, to + 32, d, us);
            }
            la::tmem_wait_st();
            bound = finite(fmaf(64.0f * k_most, ud_most, fmaf(64.0f * head->most_q, 16384.0f / dqs, r_most * (keep + fabsf(by)))));
            arrive(&s_u);
            if (!SUM) {
                s_xm[half][pl] = max_abs<32>(x);
                pair_sync();
                const float xi = scale_of(max_over(s_xm));
                if (half == 0) s_xsc[ph][pl] = xi;
                const uint32_t to = tm + my + bD1 + 16 * half;
                put2(to, to + 32, x, xi);
                la::tmem_wait_st();
                arrive(&s_xi);
            }
            ok = ok && wait(&s_d3, ph, &s_fail);
            la::tc_fence_after();
            arrive(&s_free[ph]);
#pragma unroll
            for (int c = 0; c < NB; c++) {
                la::tmem_ld32(tm + my + bD3 + half * W + 32 * c, d);
#pragma unroll
                for (int n = 0; n < 32; n += 2) {
                    const float2 f = fma2(splat2(inv3), make_float2(d[n], d[n + 1]), make_float2(R[32 * c + n], R[32 * c + n + 1]));
                    R[32 * c + n] = f.x;
                    R[32 * c + n + 1] = f.y;
                }
            }
        }
        if (mine && ok && (SUM || (r.last && seg == 0))) {
            float* to = SUM ? seg_state : r.last + bh * a.N * a.P;
#pragma unroll
            for (int n = 0; n < W; n++)
                if (half * W + n < a.N) to[(half * W + n) * a.P + p] = R[n];
        }
    } else if (warp < kStateThreads / 32 + 4) {
        leave_regs<112>();
        const bool first = tid == kStateThreads;
        Ring ring = {staging, 0};
        for (int i = 0; i < chunks; i++) {
            const uint32_t ph = i & 1;
            const int64_t image = images + chunk_of(i);
            char* at = sm + ph * L::bytes;
            const ImageHead* head = reinterpret_cast<const ImageHead*>(at + L::head);
            const float dy_scale = a.scale * r.dy_inv[image];
            wait(&s_full[ph], (i >> 1) & 1, &s_fail);
            auto scaled = [&](int hf, float (&z)[32]) {  // scale e^c dY of 32 tokens
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const uint4 v = *unit(at + L::dy, pl, 4 * hf + u);
                    const uint32_t y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float2 f = mul2(mul2(splat2(dy_scale), *reinterpret_cast<const float2*>(&head->up[32 * hf + 8 * u + 2 * e])), unpack2<__half>(y[e]));
                        z[8 * u + 2 * e] = f.x;
                        z[8 * u + 2 * e + 1] = f.y;
                    }
                }
            };
            {
                float z[2][32];
                scaled(0, z[0]);
                scaled(1, z[1]);
                arrive(&s_free[ph]);
                const float dqs = scale_of(fmaxf(max_abs<32>(z[0]), max_abs<32>(z[1])));
                s_dqs[ph][pl] = dqs;
                if (i > 0) wait(&s_dq, ph ^ 1, &s_fail);  // the last parts are used
                la::tc_fence_after();
                put2(tm + my + bDq, tm + my + bDq + 32, z[0], dqs);
                put2(tm + my + bDq + 16, tm + my + bDq + 48, z[1], dqs);
            }
            la::tmem_wait_st();
            arrive(&s_dyq);
            if (SUM) continue;
            // R's and X's parts under one scale each: what the largest channel's is
            wait(&s_r, ph, &s_fail);
            la::tc_fence_after();
            uint32_t x[32], z[32];
            float own = s_rs[ph][pl], all = group_min(own, s_red, 5);
            uint32_t f = pack2<__half>(all / own, all / own);
            if (first) r.state_inv[image] = 1.0f / all;
#pragma unroll 1
            for (int c = 0; c < 2 * NB; c++) {
                tmem_bits(tm + my + bR + 32 * c, x);
                if (c == 2 * NB - 1) arrive(&s_early);
                ring.put(x, f, r.states + image * state_bytes(NB) + c * kPieceBytes);
            }
            wait(&s_xi, ph, &s_fail);
            la::tc_fence_after();
            own = s_xsc[ph][pl], all = group_min(own, s_red, 5);
            f = pack2<__half>(all / own, all / own);
            if (first) r.x_inv[image] = 1.0f / all;
            tmem_bits(tm + my + bD1, x);
            tmem_bits(tm + my + bD1 + 32, z);
            arrive(&s_late);
            ring.put(x, f, r.xs + image * kRowsBytes);
            ring.put(z, f, r.xs + image * kRowsBytes + kPieceBytes);
        }
        if (first) la::bulk_wait_all();
    } else {
        leave_regs<56>();
        const int role = __shfl_sync(kFull, warp, 0) - (kThreads - 128) / 32, steps = __shfl_sync(kFull, chunks, 0);
        if (role == 1 && (tid & 31) == 0) {  // loads
            auto image = [&](int i) { return w.images + (bh * w.chunks + chunk_of(i)) * kImageBytes; };
            auto grows = [&](int i) { return i < chunks ? reinterpret_cast<const ImageHead*>(image(i) + 4 * kTileBytes)->grown : 0; };
            int grown = grows(0);
            for (int i = 0; i < chunks; i++) {
                const int next = grows(i + 1);  // (on its way while the stage is waited for)
                if (i > 1 && !wait(&s_free[i & 1], ((i >> 1) + 1) & 1, &s_fail)) break;
                char* at = sm + (i & 1) * L::bytes;
                uint64_t* bar = &s_full[i & 1];
                const int ch = chunk_of(i);
                mbar_expect_tx(bar, NB * L::block + 6 * kTileBytes + (int)sizeof(ImageHead));
                bulk_load(at, w.keys + ((b * w.chunks + ch) * a.G + hq) * (NB * 2 * kTileBytes), NB * L::block, bar);
                bulk_load(at + L::dy, r.dys + (images + ch) * kPieceBytes, kPieceBytes, bar);
                if (!grown) {
                    bulk_load(at + L::image, image(i), kImageBytes, bar);
                } else {
                    const char* turned = r.turned + (bh * w.chunks + ch) * kTurnedBytes;
                    bulk_load(at + L::image, turned, 2 * kTileBytes, bar);
                    bulk_load(at + L::image + 2 * kTileBytes, image(i) + 2 * kTileBytes, 2 * kTileBytes, bar);
                    bulk_load(at + L::head, turned + 2 * kTileBytes, (int)sizeof(ImageHead), bar);
                }
                grown = next;
            }
        } else if (role == 0) {  // products
            for (int i = 0; i < steps; i++) {
                const uint32_t ph = i & 1;
                const uint32_t at = smem_addr(sm + ph * L::bytes), M = at + L::image, P = M + 2 * kTileBytes;
                constexpr uint32_t dK = la::mma_desc<__half>(128, C, false, false), dR = la::mma_desc<__half>(128, C, false, true),
                                   dN = la::mma_desc<__half>(128, 64 * NB, false, true);
                if (!warp_wait(&s_full[ph], (i >> 1) & 1, &s_fail)) break;
                if (i > 0 && !warp_wait(&s_u, ph ^ 1, &s_fail)) break;  // D2 is read
                la::tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int part = 1; part >= 0; part--)
#pragma unroll
                        for (int s = 0; s < 4; s++)
                            la::mma(tm + bD0, la::smem_desc(at + L::dy + s * 32), la::smem_desc(P + part * kTileBytes + s * 2048), dR, part < 1 || s > 0);
                }
                if (!SUM && i > 0 && !warp_wait(&s_late, ph ^ 1, &s_fail)) break;  // X has left D1's columns
                if (!warp_wait(&s_r, ph, &s_fail)) break;
                la::tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int part = 1; part >= 0; part--)
#pragma unroll
                        for (int s = 0; s < 4 * NB; s++)
                            la::mma_ts(tm + bD1, tm + bR + part * 32 * NB + 8 * s, la::smem_desc(at + (s >> 2) * L::block + (s & 3) * 32), dK, part < 1 || s > 0);
                    la::mma_commit(&s_d1);
                }
                if (!warp_wait(&s_dyq, ph, &s_fail)) break;
                la::tc_fence_after();
                auto update = [&](uint32_t left, uint32_t keys) {  // two parts
#pragma unroll
                    for (int part = 1; part >= 0; part--)
#pragma unroll
                        for (int s = 0; s < 4; s++)
                            la::mma_ts(tm + bD3, tm + left + part * 32 + 8 * s, la::smem_desc(keys + s * 2048, L::block), dN, part < 1 || s > 0);
                };
                if (elect()) {
                    update(bDq, at + kTileBytes);
                    la::mma_commit(&s_dq);
                }
                if (!warp_wait(&s_x, ph, &s_fail)) break;
                la::tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int o = 0; o < 3; o++)  // lo hi, hi lo, hi hi
#pragma unroll
                        for (int s = 0; s < 4; s++)
                            la::mma_ts(tm + bD0, tm + bX + (o == 0 ? 32 : 0) + 8 * s, la::smem_desc(M + (o == 1 ? kTileBytes : 0) + s * 2048), dR, o > 0 || s > 0);
                    la::mma_commit(&s_d2);
                }
                if (!warp_wait(&s_u, ph, &s_fail)) break;
                la::tc_fence_after();
                if (elect()) {
                    update(bX, at);
                    la::mma_commit(&s_d3);
                }
            }
        }
    }
    __syncwarp();
    uint64_t* const bars[6] = {&s_full[0], &s_full[1], &s_d1, &s_dq, &s_d2, &s_d3};
    la::end_block(&s_fail, w.status, bars, tm, 512);
}

// Both of the backward's walks: neither needs the other, and together they fill more SMs.
template <typename T, int NB>
__global__ void __launch_bounds__(kThreads, 1) k_walks(const __grid_constant__ TcWalkArgs w, const __grid_constant__ TcBackArgs r, int forward) {
    extern __shared__ __align__(1024) char sm[];
    if ((int)blockIdx.x < forward) walk<T, NB, kTcKeep>(w, sm);
    else walk_back<NB, false>(w, r, blockIdx.x - forward, sm);
}
// blockIdx.y: E, Phi, E'
template <typename T, int NB>
__global__ void __launch_bounds__(kThreads, 1) k_sums(const __grid_constant__ TcWalkArgs w, const __grid_constant__ TcBackArgs r) {
    extern __shared__ __align__(1024) char sm[];
    if (blockIdx.y < 2) walk<T, NB, kTcSum>(w, sm);
    else walk_back<NB, true>(w, r, blockIdx.x, sm);
}

// S <- Phi S + E over the segments, from h0; seg_state receives the state each segment starts
// from.  blockIdx.y 1: R <- Phi^T R + E' from the last.  A block: 8 columns of one head's state, in shared memory.  Warp w takes the terms of states w, w + 8, ..: a lane
// four rows and all columns; the warps' sums are added in order.  The next Phi (transposed) is on its way while one is
// used.  Bound by reading shared memory.  65536 tokens, 8 heads, 18 segments: 50 us (sums over states in single threads, 19 segments: 86).
constexpr int kCarryCols = 8;
__global__ void __launch_bounds__(256) k_carry(TcWalkArgs w, TcBackArgs r) {
    extern __shared__ __align__(16) float phi[];  // [2][N][N], then the warps' sums [8][N][8]
    __shared__ __align__(16) float s[la::kMaxN][kCarryCols];
    __shared__ __align__(8) uint64_t s_full[2];
    __shared__ uint32_t s_fail;
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = (int)a.N, n = tid >> 1, c = (tid & 1) * 4;
    const int64_t ptiles = (a.P + kCarryCols - 1) / kCarryCols, p0 = blockIdx.x % ptiles * kCarryCols, bh = blockIdx.x / ptiles;
    const bool back = blockIdx.y == 1;
    const float *phis = back ? w.seg_phi_t : w.seg_phi, *init = back ? r.init : w.init;
    float* const states = back ? r.seg_state : w.seg_state;
    const int K = (int)w.plan.K;
    auto segment = [&](int k) { return bh * K + (back ? K - 1 - k : k); };
    float* sums = phi + 2 * N * N;
    if (tid == 0) {
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        s_fail = 0;
        fence_proxy_async_smem();
    }
    auto load = [&](int k) {
        mbar_expect_tx(&s_full[k & 1], N * N * 4);
        bulk_load(phi + (k & 1) * N * N, phis + segment(k) * N * N, N * N * 4, &s_full[k & 1]);
    };
    const bool mine = n < N;  // (P is a multiple of 8)
    float4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (mine && init) x = *reinterpret_cast<const float4*>(init + (bh * N + n) * a.P + p0 + c);
    __syncthreads();
    if (tid == 0) load(0);
    for (int k = 0; k < K; k++) {
        float4* at = reinterpret_cast<float4*>(states + (segment(k) * N + n) * a.P + p0 + c);
        float4 e = {0.0f, 0.0f, 0.0f, 0.0f};
        if (mine) {
            if (k + 1 < K) e = *at;
            *reinterpret_cast<float4*>(&s[n][c]) = x;
            *at = x;
        }
        if (k + 1 == K) break;
        __syncthreads();  // (the Phi before is used)
        if (tid == 0 && k + 2 < K) load(k + 1);
        wait(&s_full[k & 1], (k >> 1) & 1, &s_fail);
        const float* f = phi + (k & 1) * N * N;
        float2 y[4][kCarryCols / 2] = {};  // rows 4 lane ..
        if (4 * lane < N)
#pragma unroll 4
            for (int m = warp; m < N; m += 8) {
                const float4 p = *reinterpret_cast<const float4*>(f + m * N + 4 * lane), z0 = *reinterpret_cast<const float4*>(&s[m][0]),
                             z1 = *reinterpret_cast<const float4*>(&s[m][4]);
                const float ps[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    y[r][0] = fma2(splat2(ps[r]), make_float2(z0.x, z0.y), y[r][0]);
                    y[r][1] = fma2(splat2(ps[r]), make_float2(z0.z, z0.w), y[r][1]);
                    y[r][2] = fma2(splat2(ps[r]), make_float2(z1.x, z1.y), y[r][2]);
                    y[r][3] = fma2(splat2(ps[r]), make_float2(z1.z, z1.w), y[r][3]);
                }
            }
        if (4 * lane < N)
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int j = 0; j < 4; j += 2)
                    *reinterpret_cast<float4*>(sums + (warp * N + 4 * lane + r) * kCarryCols + 2 * j) = make_float4(y[r][j].x, y[r][j].y, y[r][j + 1].x, y[r][j + 1].y);
        __syncthreads();
        if (mine) {
            x = e;
#pragma unroll
            for (int u = 0; u < 8; u++) {
                const float4 z = *reinterpret_cast<const float4*>(sums + (u * N + n) * kCarryCols + c);
                x = make_float4(x.x + z.x, x.y + z.y, x.z + z.z, x.w + z.w);
            }
        }
    }
    __syncthreads();
    if (tid == 0 && s_fail) {
        atomicOr(w.status, kDevWaitTimeout);
        for (int i = 0; i < 2; i++)
            for (uint32_t ph = 0; ph < 2; ph++) mbar_wait(&s_full[i], ph, la::kDrainLimitNs);
    }
}

template <typename T, int NB, TcWalkMode MODE> cudaError_t walk_go(const TcWalkArgs& w, cudaStream_t st) {
    constexpr int bytes = 2 * Stage<NB, MODE == kTcY>::bytes +
                          (MODE == kTcY ? 2 * kTileBytes : 0);
    const cudaError_t e = la::allow_smem<k_walk<T, NB, MODE>>(bytes);
    if (e != cudaSuccess) return e;
    const int64_t segs = MODE == kTcSum ? w.plan.K - 1 : w.plan.K;
    const dim3 grid((unsigned)(ceil_div(w.a.P, kTileP) * w.a.Bsz * w.a.H * segs), MODE == kTcSum ? 2 : 1);
    k_walk<T, NB, MODE><<<grid, kThreads, bytes, st>>>(w);
    return cudaGetLastError();
}
template <typename T, int NB> cudaError_t walks_go(const TcWalkArgs& w, const TcBackArgs& r, cudaStream_t st) {
    constexpr int keep = 2 * Stage<NB, false>::bytes, back = 2 * BackStage<NB>::bytes, bytes = (keep > back ? keep : back) + kRing * kPieceBytes;
    const cudaError_t e = la::allow_smem<k_walks<T, NB>>(bytes);
    if (e != cudaSuccess) return e;
    const int64_t units = ceil_div(w.a.P, kTileP) * w.a.Bsz * w.a.H * w.plan.K;
    k_walks<T, NB><<<(unsigned)(2 * units), kThreads, bytes, st>>>(w, r, (int)units);
    return cudaGetLastError();
}
template <typename T, int NB> cudaError_t sums_go(const TcWalkArgs& w, const TcBackArgs& r, cudaStream_t st) {
    constexpr int fwd = 2 * Stage<NB, false>::bytes, back = 2 * BackStage<NB>::bytes, bytes = fwd > back ? fwd : back;
    const cudaError_t e = la::allow_smem<k_sums<T, NB>>(bytes);
    if (e != cudaSuccess) return e;
    k_sums<T, NB><<<dim3((unsigned)(ceil_div(w.a.P, kTileP) * w.a.Bsz * w.a.H * w.plan.K), 3), kThreads, bytes, st>>>(w, r);
    return cudaGetLastError();
}
template <typename T, int NB> cudaError_t walk_mode(const TcWalkArgs& w, TcWalkMode mode, cudaStream_t st) {
    if (mode == kTcSum) return walk_go<T, NB, kTcSum>(w, st);
    return walk_go<T, NB, kTcY>(w, st);
}

}  // namespace

cudaError_t launch_tc_walk(const TcWalkArgs& w, TcWalkMode mode, cudaStream_t st) {
    if (w.a.dtype == 1) return w.a.N <= 64 ? walk_mode<__half, 1>(w, mode, st) : walk_mode<__half, 2>(w, mode, st);
    return w.a.N <= 64 ? walk_mode<__nv_bfloat16, 1>(w, mode, st) : walk_mode<__nv_bfloat16, 2>(w, mode, st);
}

cudaError_t launch_tc_walks(const TcWalkArgs& w, const TcBackArgs& r, cudaStream_t st) {
    if (w.a.dtype == 1) return w.a.N <= 64 ? walks_go<__half, 1>(w, r, st) : walks_go<__half, 2>(w, r, st);
    return w.a.N <= 64 ? walks_go<__nv_bfloat16, 1>(w, r, st) : walks_go<__nv_bfloat16, 2>(w, r, st);
}

cudaError_t launch_tc_sums(const TcWalkArgs& w, const TcBackArgs& r, cudaStream_t st) {
    if (w.a.dtype == 1) return w.a.N <= 64 ? sums_go<__half, 1>(w, r, st) : sums_go<__half, 2>(w, r, st);
    return w.a.N <= 64 ? sums_go<__nv_bfloat16, 1>(w, r, st) : sums_go<__nv_bfloat16, 2>(w, r, st);
}

cudaError_t launch_tc_carry(const TcWalkArgs& w, const TcBackArgs* r, cudaStream_t st) {
    const int N = (int)w.a.N, bytes = (2 * N * N + 8 * N * kCarryCols) * 4;
    const cudaError_t e = la::allow_smem<k_carry>((2 * la::kMaxN * la::kMaxN + 8 * la::kMaxN * kCarryCols) * 4);
    if (e != cudaSuccess) return e;
    k_carry<<<dim3((unsigned)(ceil_div(w.a.P, kCarryCols) * w.a.Bsz * w.a.H), r ? 2 : 1), 256, bytes, st>>>(w, r ? *r : TcBackArgs{});
    return cudaGetLastError();
}

}  // namespace gdr
}  // namespace ss
