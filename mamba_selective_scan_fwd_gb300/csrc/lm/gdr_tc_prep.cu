// Gated delta rule on the tensor cores: what a chunk's products need that does not
// depend on the state, for all chunks at once.
//
// One block: one chunk of the heads that share a head of q and k.  [K; Q] K^T is one
// product of 128 rows.  Per head A = beta e^{c_i - c_j} k_i . k_j below the diagonal;
// M = (I + A)^{-1} in f32 by forward substitution, in blocks (not by a series in A, whose
// powers may be large where M is not).  4 x 4096 tokens, 32 heads in 16 groups, N = 128: 137 us, of which its 134 MB read and 420
// written are 82.  One head at a time in a block of four warps: a block's
// steps wait for one another, and four blocks on an SM cover that.
#include "gdr_tc.h"
#include "../simd.cuh"
#include "tc.cuh"
#include "gdr_dev.cuh"

namespace ss {
namespace gdr {
namespace {

using la::Two;
using la::two_diff;
using la::unit;
using la::pack2;
using la::unpack2;
using bf16 = __nv_bfloat16;

constexpr int C = kChunk;
constexpr int LDA = C + 4;
constexpr int kThreads = 128, kHeads = 4;  // heads whose decays are made at a time: one a warp

// K and Q as they come; then the image as it goes
template <int NB> struct PrepSmem {
    static constexpr int kq = 0, image = 0, first = NB * 16384 > kImageBytes ? NB * 16384 : kImageBytes, a = first,
                         total = a + C * LDA * 4;
};

// 16 values times s as two f16 parts, in units u0, u0 + 1 of a row of two tiles
__device__ __forceinline__ void put_parts(char* hi, char* lo, int row, int u0, const float* x, float s) {
#pragma unroll
    for (int u = 0; u < 2; u++) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float2 f = mul2(make_float2(x[8 * u + 2 * i], x[8 * u + 2 * i + 1]), splat2(s));
            h[i] = pack2<__half>(f.x, f.y);
            f = fma2(unpack2<__half>(h[i]), splat2(-1.0f), f);
            l[i] = pack2<__half>(f.x, f.y);
        }
        *unit(hi, row, u0 + u) = make_uint4(h[0], h[1], h[2], h[3]);
        *unit(lo, row, u0 + u) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

__device__ __forceinline__ float warp_max(float v) {  // v >= 0
    uint32_t m;
    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(__float_as_uint(v)));
    return __uint_as_float(m);
}
__device__ __forceinline__ float max4(const float* x) { return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])); }

// A value as two tf32 parts (22 bits).
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// One warp: 16 x 16 of left right, n terms (a multiple of 8), operands in two tf32 parts.  (A warp's matrix instruction, because
// such a product is too small for a tensor-memory one and its operands are f32 in shared memory, whose reads
// bound this kernel: as products of four by two values a thread it took four times the reads; 4 x 4096 tokens, 32 heads, P in
// one part: 133 us so, 127 with it.)
__device__ __forceinline__ void product16(const float* left, const float* right, int n, float (&out)[2][4]) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) out[j][e] = 0.0f;
#pragma unroll 2
    for (int k = 0; k < n; k += 8) {
        uint32_t ah[4], al[4];
#pragma unroll
        for (int e = 0; e < 4; e++) split_tf32(left[(g + 8 * (e & 1)) * LDA + k + t + 4 * (e >> 1)], ah[e], al[e]);
#pragma unroll
        for (int j = 0; j < 2; j++) {
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int e = 0; e < 2; e++) split_tf32(right[(k + t + 4 * e) * LDA + 8 * j + g], bh[e], bl[e]);
            mma_tf32(out[j], al, bh);
            mma_tf32(out[j], ah, bl);
            mma_tf32(out[j], ah, bh);
        }
    }
}
__device__ __forceinline__ void put16(float* to, const float (&x)[2][4], float sign) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
        for (int r = 0; r < 2; r++)
            *reinterpret_cast<float2*>(to + (g + 8 * r) * LDA + 8 * j + 2 * t) = make_float2(sign * x[j][2 * r], sign * x[j][2 * r + 1]);
}

// A (64 x 64, below the diagonal; zeros elsewhere) becomes M = (I + A)^{-1} in place, four warps: blocks of 16 by
// forward substitution (a thread a column), then [[a, 0], [A, b]]: -b A a, of 16 and of 32.
__device__ __forceinline__ void invert(float* A) {
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid < C) {
        const int d = tid & ~15, j = tid & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; i++) {
            float s0 = i == j ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
            for (int k = 0; k < i; k += 4) {
                const float4 r = *reinterpret_cast<const float4*>(A + (d + i) * LDA + d + k);
                s0 = fmaf(-r.x, x[k], s0);
                if (k + 1 < i) s1 = fmaf(-r.y, x[k + 1], s1);
                if (k + 2 < i) s0 = fmaf(-r.z, x[k + 2], s0);
                if (k + 3 < i) s1 = fmaf(-r.w, x[k + 3], s1);
            }
            x[i] = s0 + s1;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; i++) A[(d + i) * LDA + d + j] = x[i];
        __syncwarp();
        float t[2][4];  // warp w: the block below the diagonal's, between its two
        float *a = A + 32 * warp * (LDA + 1), *below = a + 16 * LDA;
        product16(below, a, 16, t);
        __syncwarp();
        put16(below, t, 1.0f);
        __syncwarp();
        product16(below + 16, below, 16, t);
        __syncwarp();
        put16(below, t, -1.0f);
    }
    __syncthreads();
    const int r = 16 * (warp >> 1), c = 16 * (warp & 1);  // warp: a block of the lower left 32 x 32
    float* quarter = A + 32 * LDA;
    float t[2][4];
    product16(quarter + r * LDA + c, A + c * LDA + c, 32 - c, t);  // (a is zero above its blocks' diagonal)
    __syncthreads();
    put16(quarter + r * LDA + c, t, 1.0f);
    __syncthreads();
    product16(quarter + r * LDA + 32, quarter + c, 16 + r, t);
    __syncthreads();
    put16(quarter + r * LDA + c, t, -1.0f);
    __syncthreads();
}

template <typename T, int NB>
__global__ void __launch_bounds__(kThreads, 4) k_prep(const __grid_constant__ PrepArgs w) {
    extern __shared__ __align__(1024) char sm[];
    using L = PrepSmem<NB>;
    __shared__ __align__(8) uint64_t s_ld, s_mma;
    __shared__ uint32_t s_tm, s_fail;
    __shared__ Two s_c[kHeads][C];
    __shared__ __align__(16) float s_tail[kHeads][C];  // e^{c_e - c_t}, e the end of the token's run of 16
    __shared__ float s_beta[kHeads][C], s_max[2][4];
    __shared__ la::Decay s_by[kHeads];
    __shared__ bool s_flat[kHeads];  // no run of 16 leaves 2^-64 .. 2^64
    __shared__ int8_t s_grow[kHeads][C], s_rise[kHeads][C];
    __shared__ bool s_grown[kHeads];
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned id = blockIdx.x;
    const int split = id % w.splits;
    id /= w.splits;
    const int gq = id % (unsigned)a.G;
    id /= (unsigned)a.G;
    const int64_t chunk = id % (unsigned)w.chunks, b = id / (unsigned)w.chunks, t0 = chunk * C;
    const int rep = (int)(a.H / a.G), h_lo = gq * rep + rep * split / w.splits, h_hi = gq * rep + rep * (split + 1) / w.splits;
    const int nv = (int)max((int64_t)0, min((int64_t)C, row_length(a, b) - t0));
    if (nv == 0) return;  // no walk gets here
    // this warp's head of the first few: what its decays come from, on its way before all else
    float g[2], beta_t[2];
    auto fetch = [&](int h) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int t = 2 * lane + i;
            g[i] = beta_t[i] = 0.0f;
            if (t < nv && h < h_hi) {
                if (a.g) g[i] = a.g[(b * a.L + t0 + t) * a.H + h];
                beta_t[i] = a.beta[(b * a.L + t0 + t) * a.H + h];
            }
        }
    };
    fetch(h_lo + warp);
    char *KQ = sm + L::kq, *I = sm + L::image;
    float* A = reinterpret_cast<float*>(sm + L::a);
    ImageHead* head = reinterpret_cast<ImageHead*>(I + 4 * kTileBytes);
    if (tid == 0) {
        mbar_init(&s_ld, 1);
        mbar_init(&s_mma, 1);
        s_fail = 0;
        fence_proxy_async_smem();
        mbar_expect_tx(&s_ld, NB * 16384);
#pragma unroll
        for (int n = 0; n < NB; n++) {
            la::tma_load_4d(KQ + n * 16384, &w.k, n * 64, (int)gq, (int)t0, (int)b, &s_ld);
            la::tma_load_4d(KQ + n * 16384 + kTileBytes, &w.q, n * 64, (int)gq, (int)t0, (int)b, &s_ld);
        }
    }
    if (warp == 1) la::tmem_alloc(&s_tm, 64);
    auto decays = [&] {  // this warp's head
        const float x[2] = {la::clamp_g(g[0]) * la::kLog2e, la::clamp_g(g[1]) * la::kLog2e};
        bool flat;
        const Pair p = chunk_decays(x, s_c[warp], s_tail[warp], flat);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            s_beta[warp][2 * lane + i] = beta_t[i];
            s_grow[warp][2 * lane + i] = (int8_t)p.grow[i];
            s_rise[warp][2 * lane + i] = (int8_t)p.rise[i];
        }
        const bool grown = __any_sync(kFull, p.grow[0] | p.grow[1] | p.rise[0] | p.rise[1]);
        if (lane == 0) {
            s_flat[warp] = flat;
            s_grown[warp] = grown;
        }
        // the chunk's decay, in natural units from the same sum (rounded once more: 2^-24 of cl)
        if (lane == 31) s_by[warp] = la::decay_of((p.sum.h + p.sum.l) * kLn2);
    };
    if (h_lo + warp < h_hi) decays();
    __syncthreads();
    la::tc_fence_after();
    const uint32_t tm = s_tm, my = (uint32_t)(tid & 96) << 16;
    bool ok = la::wait_or_fail(&s_ld, 0, &s_fail);
    if (tid == 0 && ok) {
        constexpr uint32_t d = la::mma_desc<T>(128, 64, false, false);
        const uint32_t at = smem_addr(KQ);
#pragma unroll
        for (int s = 0; s < 4 * NB; s++) {
            const uint32_t x = at + (s >> 2) * 16384 + (s & 3) * 32;
            la::mma(tm, la::smem_desc(x), la::smem_desc(x), d, s > 0);
        }
        la::mma_commit(&s_mma);
    }
    __syncwarp();
    // K and Q as f16: unit tid + 128 i of the 512 of each tile
    float scale_k, scale_q, most_k, most_q;
    {
        uint4 x[2][4 * NB];
        float most[2] = {};
#pragma unroll
        for (int side = 0; side < 2; side++)
#pragma unroll
            for (int i = 0; i < 4 * NB; i++) {
                const int at = tid + 128 * (i & 3);
                uint4& y = x[side][i];
                y = *reinterpret_cast<const uint4*>(KQ + (i >> 2) * 16384 + side * kTileBytes + at * 16);
                if (at >> 3 >= nv) y = make_uint4(0, 0, 0, 0);
                const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float2 f = unpack2<T>(v[e]);
                    most[side] = fmaxf(most[side], fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
#pragma unroll
        for (int side = 0; side < 2; side++) {
            const float m = warp_max(most[side]);
            if (lane == 0) s_max[side][warp] = m;
        }
        __syncthreads();
        most_k = max4(s_max[0]);
        most_q = max4(s_max[1]);
        scale_k = la::f16_scale(most_k);
        scale_q = la::f16_scale(most_q);
        char* keys = w.keys + ((b * w.chunks + chunk) * a.G + gq) * (NB * 16384);
        if (split == 0)
#pragma unroll
            for (int side = 0; side < 2; side++)
#pragma unroll
                for (int i = 0; i < 4 * NB; i++) {
                    const uint4& y = x[side][i];
                    const uint32_t v[4] = {y.x, y.y, y.z, y.w};
                    const float2 scale = splat2(side ? scale_q : scale_k);
                    uint32_t r[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float2 f = mul2(unpack2<T>(v[e]), scale);
                        r[e] = pack2<__half>(f.x, f.y);
                    }
                    *reinterpret_cast<uint4*>(keys + (i >> 2) * 16384 + side * kTileBytes + (tid + 128 * (i & 3)) * 16) = make_uint4(r[0], r[1], r[2], r[3]);
                }
    }
    ok = la::wait_or_fail(&s_mma, 0, &s_fail) && ok;
    la::tc_fence_after();
    for (int h0 = h_lo; h0 < h_hi; h0 += kHeads) {
        if (h0 > h_lo) {
            fetch(h0 + warp);
            __syncthreads();
            if (h0 + warp < h_hi) decays();
        }
        for (int h = h0; h < min(h_hi, h0 + kHeads); h++) {
            const int hl = h - h0;
            if (__syncthreads_or(!ok)) break;  // (and: the last head's image has left, s_max is free)
            // thread: row i of K K^T (warps 0, 1) or Q K^T
            const bool is_q = tid >= C;
            const int i = tid & 63, last = is_q ? i : i - 1;
            float s[C];
            la::tmem_ld32(tm + my, *reinterpret_cast<float(*)[32]>(s));
            la::tmem_ld32(tm + my + 32, *reinterpret_cast<float(*)[32]>(s + 32));
            const Two ci = s_c[hl][i];
            const float f = is_q ? 1.0f : s_beta[hl][i];
            pair_factors(s, s_c[hl], s_tail[hl], s_flat[hl], 0, ci, f, last);
            if (i >= nv)  // (whatever the row holds)
#pragma unroll
                for (int j = 0; j < C; j++) s[j] = 0.0f;
            const bool turned = w.turned && s_grown[hl];
            float most = 0.0f;
            if (is_q) {
                if (turned)
#pragma unroll
                    for (int j = 0; j < C; j++) s[j] *= power2(s_rise[hl][i] - s_rise[hl][j]);
#pragma unroll
                for (int j = 0; j < C; j++) most = fmaxf(most, fabsf(s[j]));
                most = warp_max(most);
            } else {
#pragma unroll
                for (int j = 0; j < C; j += 4)
                    *reinterpret_cast<float4*>(A + i * LDA + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
            }
            if (lane == 0) s_max[0][warp] = most;
            if (tid < C) {
                const Two c = s_c[hl][tid], cl = s_c[hl][C - 1];
                const float up = ex2a(c.h + c.l);
                head->up[tid] = up;
                head->beta_up[tid] = s_beta[hl][tid] * up;
                head->down[tid] = ex2a(two_diff(cl, c)) * power2(s_grow[hl][C - 1]);
                head->beta[tid] = s_beta[hl][tid] * power2(-s_grow[hl][tid]);
                head->grow[tid] = __float2bfloat16(power2(s_grow[hl][tid]));
                head->rise[tid] = s_rise[hl][tid];
                head->tail[tid] = s_tail[hl][tid];
                head->c[tid] = make_float2(c.h, c.l);
            }
            __syncthreads();
            const float scale_p = la::f16_scale(fmaxf(s_max[0][2], s_max[0][3]));
            if (is_q) {
                char* hi = I + 2 * kTileBytes;
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    put_parts(hi, hi + kTileBytes, i, 2 * u, s + 16 * u, scale_p);
                    __syncwarp();  // (units in turn: the parts of all of them at once are spilled, 4 x 4096 tokens, 32 heads 138 us for 133)
                }
            }
            invert(A);
            {
                const int i = tid >> 1, j0 = (tid & 1) * 32;
                float x[32], most = 0.0f;
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(A + i * LDA + j0 + e);
                    x[e] = v.x;
                    x[e + 1] = v.y;
                    x[e + 2] = v.z;
                    x[e + 3] = v.w;
                    most = fmaxf(most, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
                }
                most = warp_max(most);
                if (lane == 0) s_max[1][warp] = most;
                __syncthreads();
                const float most_m = max4(s_max[1]), scale_m = la::f16_scale(most_m);
                put_parts(I, I + kTileBytes, i, j0 / 8, x, scale_m);
                put_parts(I, I + kTileBytes, i, j0 / 8 + 2, x + 16, scale_m);
                if (tid == 0) {
                    head->by = s_by[hl].by;
                    head->weak = s_by[hl].weak;
                    head->flat = s_flat[hl];
                    head->grown = s_grown[hl];
                    head->inv_k = 1.0f / scale_k;
                    head->inv_q = 1.0f / scale_q;
                    head->inv_m = 1.0f / scale_m;
                    head->inv_p = 1.0f / scale_p;
                    head->most_k = most_k;
                    head->most_q = most_q;
                    head->most_m = most_m;
                }
            }
            fence_proxy_async_smem();
            __syncthreads();
            if (tid == 0) {
                la::bulk_store(w.images + ((b * a.H + h) * w.chunks + chunk) * kImageBytes, I, kImageBytes);
                la::bulk_commit();
                if (turned || h + 1 < h_hi) la::bulk_wait_read();
            }
            if (turned) {  // M and the factors in the adjoints' units
                __syncthreads();
                if (tid < C) {
                    const float by = power2(s_rise[hl][tid]);
                    head->up[tid] *= by;
                    head->beta_up[tid] *= by;
                    head->down[tid] *= power2(-s_rise[hl][tid]);
                }
                const int i = tid >> 1, j0 = (tid & 1) * 32;
                float most = 0.0f;
#pragma unroll 1
                for (int j = j0; j < j0 + 32; j++) {
                    float& x = A[i * LDA + j];
                    x *= power2(s_rise[hl][i] - s_rise[hl][j]);
                    most = fmaxf(most, fabsf(x));
                }
                most = warp_max(most);
                if (lane == 0) s_max[1][warp] = most;
                __syncthreads();
                const float most_m = max4(s_max[1]), scale_m = la::f16_scale(most_m);
#pragma unroll 1
                for (int j = j0; j < j0 + 32; j += 16) put_parts(I, I + kTileBytes, i, j / 8, A + i * LDA + j, scale_m);
                if (tid == 0) {
                    head->inv_m = 1.0f / scale_m;
                    head->most_m = most_m;
                }
                fence_proxy_async_smem();
                __syncthreads();
                if (tid == 0) {
                    char* to = w.turned + ((b * a.H + h) * w.chunks + chunk) * kTurnedBytes;
                    la::bulk_store(to, I, 2 * kTileBytes);
                    la::bulk_store(to + 2 * kTileBytes, head, sizeof(ImageHead));
                    la::bulk_commit();
                    if (h + 1 < h_hi) la::bulk_wait_read();
                }
            }
        }
    }
    if (tid == 0) la::bulk_wait_all();
    uint64_t* const bars[2] = {&s_ld, &s_mma};
    la::end_block(&s_fail, w.status, bars, tm, 64);
}

// dY's image: 64 tokens of 128 value channels of one head, transposed, in the adjoints' units, f16 under the scale of its largest
// value; tokens past the row's length zero.  Bound by HBM (2 x 4096 tokens, 32 heads of 128: 30 us, copying 20).
template <typename T> __global__ void __launch_bounds__(256, 8) k_dy(Args a, int64_t chunks, const char* images, char* dys, float* dy_inv) {
    constexpr int LD = 132;  // (a row's 16-byte units spread over the banks)
    __shared__ __align__(16) T s[C][LD];
    __shared__ float s_max[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t ptiles = (a.P + 127) / 128;
    int64_t id = blockIdx.x;
    const int64_t chunk = id % chunks;
    id /= chunks;
    const int64_t p0 = id % ptiles * 128, bh = id / ptiles, b = bh / a.H, h = bh % a.H, t0 = chunk * C;
    const int nv = (int)max((int64_t)0, min((int64_t)C, row_length(a, b) - t0));
    if (nv == 0) return;
    const T* from = static_cast<const T*>(a.dy.p) + b * a.dy.batch + t0 * a.dy.token + h * a.P + p0;
    const ImageHead* head = reinterpret_cast<const ImageHead*>(images + (bh * chunks + chunk) * kImageBytes + 4 * kTileBytes);
    const bool grown = head->grown;
    auto unit_of = [&](int t) { return ldf(&head->grow[t]) * power2(-head->rise[t]); };
    float m[4] = {}, most = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int t = (tid + 256 * i) >> 4, u = tid & 15;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (t < nv && p0 + 8 * u < a.P) x = *reinterpret_cast<const uint4*>(from + t * a.dy.token + 8 * u);
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float2 f = unpack2<T>(v[e]);
            m[i] = fmaxf(m[i], fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        *reinterpret_cast<uint2*>(&s[t][8 * u]) = make_uint2(x.x, x.y);
        *reinterpret_cast<uint2*>(&s[t][8 * u + 4]) = make_uint2(x.z, x.w);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) most = fmaxf(most, grown ? m[i] * unit_of((tid + 256 * i) >> 4) : m[i]);
    most = warp_max(most);
    if (lane == 0) s_max[warp] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; i++) most = fmaxf(most, s_max[i]);
    const float scale = la::f16_scale(most);
    char* to = dys + (int64_t)blockIdx.x * kPieceBytes;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int at = tid + 256 * i, p = at >> 3, u = (at & 7) ^ (p & 7);
        uint32_t x[4];
        if (!grown) {
#pragma unroll
            for (int e = 0; e < 4; e++) x[e] = pack2<__half>(scale * ldf(&s[8 * u + 2 * e][p]), scale * ldf(&s[8 * u + 2 * e + 1][p]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int t = 8 * u + 2 * e;
                x[e] = pack2<__half>(scale * unit_of(t) * ldf(&s[t][p]), scale * unit_of(t + 1) * ldf(&s[t + 1][p]));
            }
        }
        *reinterpret_cast<uint4*>(to + at * 16) = make_uint4(x[0], x[1], x[2], x[3]);
    }
    if (tid == 0) dy_inv[blockIdx.x] = most == 0.0f ? 0.0f : 1.0f / scale;  // (zeros bound nothing)
}

template <typename T, int NB> cudaError_t prep_go(const PrepArgs& w, cudaStream_t st) {
    constexpr int bytes = PrepSmem<NB>::total;
    const cudaError_t e = la::allow_smem<k_prep<T, NB>>(bytes);
    if (e != cudaSuccess) return e;
    k_prep<T, NB><<<(unsigned)(w.a.Bsz * w.chunks * w.a.G * w.splits), kThreads, bytes, st>>>(w);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dy(const Args& a, int64_t chunks, const char* images, char* dys, float* dy_inv, cudaStream_t st) {
    const unsigned grid = (unsigned)(a.Bsz * a.H * ceil_div(a.P, kTileP) * chunks);
    if (a.dtype == 1) k_dy<__half><<<grid, 256, 0, st>>>(a, chunks, images, dys, dy_inv);
    else k_dy<bf16><<<grid, 256, 0, st>>>(a, chunks, images, dys, dy_inv);
    return cudaGetLastError();
}

cudaError_t launch_prep(const PrepArgs& w, cudaStream_t st) {
    if (w.a.dtype == 1) return w.a.N <= 64 ? prep_go<__half, 1>(w, st) : prep_go<__half, 2>(w, st);
    return w.a.N <= 64 ? prep_go<bf16, 1>(w, st) : prep_go<bf16, 2>(w, st);
}

}  // namespace gdr
}  // namespace ss
