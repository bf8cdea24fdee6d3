// Gated delta rule on the tensor cores: what a chunk's products need that does not
// depend on the state, for all chunks at once.
//
// One block: one chunk of the heads that share a head of q and k.  [K; Q] K^T is one
// product of 128 rows.  Per head A = beta e^{c_i - c_j} k_i . k_j below the diagonal;
// M = (I + A)^{-1} by blocks of 16: the diagonal ones by forward substitution (a thread a
// column), the others by distance from the diagonal, M_IJ = -M_II sum_K A_IK M_KJ, all in
// f32 (substitution, not a series in A: A's powers may be large where M is not).
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
constexpr int kHeads = 8;  // heads whose decays are made at a time: one a warp

// K and Q as they come; then the image as it goes
template <int NB, int PARTS> struct PrepSmem {
    static constexpr int kq = 0, image = 0, first = NB * 16384 > image_bytes(PARTS) ? NB * 16384 : image_bytes(PARTS), a = first,
                         m = a + C * LDA * 4, total = m + C * LDA * 4;
};

// 16 values times s as one or two f16 parts, in units u0, u0 + 1 of a row of two tiles
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
        if (lo) *unit(lo, row, u0 + u) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

__device__ __forceinline__ float warp_max(float v) {  // v >= 0
    uint32_t m;
    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(__float_as_uint(v)));
    return __uint_as_float(m);
}
__device__ __forceinline__ float max8(const float* x) {
    return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
}

// M = (I + A)^{-1} of a unit lower triangular I + A, 64 x 64, all 256 threads; M's upper
// blocks hold intermediate products and are not cleared.
__device__ __forceinline__ void invert(const float* A, float* M) {
    const int tid = threadIdx.x;
    if (tid < C) {  // diagonal blocks: thread = column
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
#pragma unroll
        for (int i = 0; i < 16; i++) M[(d + i) * LDA + d + j] = x[i];
    }
    __syncthreads();
    const int e = tid & 63, i = e >> 2, c = (e & 3) * 4;
#pragma unroll
    for (int dist = 1; dist < 4; dist++) {
        const int I = 16 * (dist + (tid >> 6)), J = I - 16 * dist;
        const bool on = (tid >> 6) < 4 - dist;
        auto product = [&](const float* left, const float* right, int n) {  // row i of left, columns c .. c + 3 of right
            float4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
            for (int k = 0; k < n; k += 4) {
                const float4 l = *reinterpret_cast<const float4*>(left + i * LDA + k);
                const float ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const float4 r = *reinterpret_cast<const float4*>(right + (k + u) * LDA + c);
                    s = make_float4(fmaf(ls[u], r.x, s.x), fmaf(ls[u], r.y, s.y), fmaf(ls[u], r.z, s.z), fmaf(ls[u], r.w, s.w));
                }
            }
            return s;
        };
        if (on) *reinterpret_cast<float4*>(M + (J + i) * LDA + I + c) = product(A + I * LDA + J, M + J * LDA + J, 16 * dist);
        __syncthreads();
        if (on) {
            const float4 s = product(M + I * LDA + I, M + J * LDA + I, 16);
            *reinterpret_cast<float4*>(M + (I + i) * LDA + J + c) = make_float4(-s.x, -s.y, -s.z, -s.w);
        }
        __syncthreads();
    }
}

template <typename T, int NB, int PARTS>
__global__ void __launch_bounds__(256, 3) k_prep(const __grid_constant__ PrepArgs w) {
    extern __shared__ __align__(1024) char sm[];
    using L = PrepSmem<NB, PARTS>;
    __shared__ __align__(8) uint64_t s_ld, s_mma;
    __shared__ uint32_t s_tm, s_fail;
    __shared__ Two s_c[kHeads][C];
    __shared__ __align__(16) float s_tail[kHeads][C];  // e^{c_e - c_t}, e the end of the token's run of 16
    __shared__ float s_beta[kHeads][C], s_max[2][8];
    __shared__ la::Decay s_by[kHeads];
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t id = blockIdx.x;
    const int64_t split = id % w.splits;
    id /= w.splits;
    const int64_t gq = id % a.G;
    id /= a.G;
    const int64_t chunk = id % w.chunks, b = id / w.chunks, t0 = chunk * C, rep = a.H / a.G;
    const int nv = (int)max((int64_t)0, min((int64_t)C, row_length(a, b) - t0));
    if (nv == 0) return;  // no walk gets here
    char *KQ = sm + L::kq, *I = sm + L::image;
    float *A = reinterpret_cast<float*>(sm + L::a), *M = reinterpret_cast<float*>(sm + L::m);
    ImageHead* head = reinterpret_cast<ImageHead*>(I + (2 + PARTS) * kTileBytes);
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
    const int64_t h_lo = gq * rep + rep * split / w.splits, h_hi = gq * rep + rep * (split + 1) / w.splits;
    auto decays = [&](int64_t h) {  // this warp's head
        float x[2], e[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int t = 2 * lane + i;
            x[i] = t < nv ? log_decay(a, b, t0 + t, h) * la::kLog2e : 0.0f;
            s_beta[warp][t] = t < nv ? a.beta[(b * a.L + t0 + t) * a.H + h] : 0.0f;
        }
        Two c[2];
        la::warp_cumsum<2>(x, c);
        const Two end = {__shfl_sync(kFull, c[1].h, lane | 7), __shfl_sync(kFull, c[1].l, lane | 7)};
#pragma unroll
        for (int i = 0; i < 2; i++) {
            s_c[warp][2 * lane + i] = c[i];
            e[i] = la::ex2(two_diff(end, c[i]));
            s_tail[warp][2 * lane + i] = e[i];
        }
        // the chunk's decay, in natural units from the same sum (rounded once more: 2^-24 of cl)
        if (lane == 31) s_by[warp] = la::decay_of((c[1].h + c[1].l) * kLn2);
    };
    if (h_lo + warp < h_hi) decays(h_lo + warp);
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
    // K (threads 0 .. 127) and Q as f16: unit u of row r of each tile; 64 x 8 NB units each
    float scale_k, scale_q;
    {
        const int mine = tid & 127, side = tid >> 7;
        float most = 0.0f;
        uint4 x[4 * NB];
#pragma unroll
        for (int i = 0; i < 4 * NB; i++) {
            const int row = (mine + 128 * i) >> 3 & 63;
            x[i] = *reinterpret_cast<const uint4*>(KQ + (i >> 2) * 16384 + side * kTileBytes + ((mine + 128 * i) & 511) * 16);
            if (row >= nv) x[i] = make_uint4(0, 0, 0, 0);
            const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float2 f = unpack2<T>(v[e]);
                most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        }
        most = warp_max(most);
        if (lane == 0) s_max[0][warp] = most;
        __syncthreads();
        scale_k = la::f16_scale(fmaxf(fmaxf(s_max[0][0], s_max[0][1]), fmaxf(s_max[0][2], s_max[0][3])));
        scale_q = la::f16_scale(fmaxf(fmaxf(s_max[0][4], s_max[0][5]), fmaxf(s_max[0][6], s_max[0][7])));
        const float2 s = splat2(side ? scale_q : scale_k);
        char* to = w.keys + ((b * w.chunks + chunk) * a.G + gq) * (NB * 16384);
        if (split == 0)
#pragma unroll
            for (int i = 0; i < 4 * NB; i++) {
                const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t r[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float2 f = mul2(unpack2<T>(v[e]), s);
                    r[e] = pack2<__half>(f.x, f.y);
                }
                *reinterpret_cast<uint4*>(to + (i >> 2) * 16384 + side * kTileBytes + ((mine + 128 * i) & 511) * 16) = make_uint4(r[0], r[1], r[2], r[3]);
            }
    }
    ok = la::wait_or_fail(&s_mma, 0, &s_fail) && ok;
    la::tc_fence_after();
    for (int64_t h0 = h_lo; h0 < h_hi; h0 += kHeads) {
        if (h0 > h_lo) {
            __syncthreads();
            if (h0 + warp < h_hi) decays(h0 + warp);
        }
        for (int64_t h = h0; h < min(h_hi, h0 + kHeads); h++) {
            const int hl = (int)(h - h0);
            if (__syncthreads_or(!ok)) break;  // (and: the last head's image has left, s_max is free)
            // thread: row i of K K^T (warps 0, 1 of a warpgroup) or Q K^T, columns j0 .. j0 + 31: two runs of 16.  A run
            // left of the row's own takes e^{c_i - c_e} e^{c_e - c_j} with e its end, the row's own an exponential each.
            const bool is_q = tid & 64;
            const int i = tid & 63, j0 = (tid >> 7) * 32, last = is_q ? i : i - 1;
            float s[32];
            la::tmem_ld32(tm + my + j0, s);
            const Two ci = s_c[hl][i];
            const float f = i >= nv ? 0.0f : is_q ? 1.0f : s_beta[hl][i];
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const int c0 = j0 + 16 * r;
                if (c0 + 16 <= (i & ~15)) {
                    const float by = f * la::ex2(two_diff(ci, s_c[hl][c0 + 15]));
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 t = *reinterpret_cast<const float4*>(&s_tail[hl][c0 + j]);
                        s[16 * r + j] *= by * t.x;
                        s[16 * r + j + 1] *= by * t.y;
                        s[16 * r + j + 2] *= by * t.z;
                        s[16 * r + j + 3] *= by * t.w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        const float e = c0 + j <= last ? la::ex2(two_diff(ci, s_c[hl][c0 + j])) : 0.0f;
                        s[16 * r + j] = c0 + j <= last ? f * e * s[16 * r + j] : 0.0f;
                    }
                }
                if (i >= nv)  // (whatever the row holds)
#pragma unroll
                    for (int j = 0; j < 16; j++) s[16 * r + j] = 0.0f;
            }
            float most = 0.0f;
            if (is_q) {
#pragma unroll
                for (int j = 0; j < 32; j++) most = fmaxf(most, fabsf(s[j]));
                most = warp_max(most);
            } else {
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<float4*>(A + i * LDA + j0 + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
            }
            if (lane == 0) s_max[0][warp] = most;
            if (tid < C) {
                const Two c = s_c[hl][tid], cl = s_c[hl][C - 1];
                const float up = la::ex2(c.h + c.l);
                head->up[tid] = up;
                head->beta_up[tid] = s_beta[hl][tid] * up;
                head->down[tid] = la::ex2(two_diff(cl, c));
                head->beta[tid] = s_beta[hl][tid];
            }
            __syncthreads();
            const float scale_p = la::f16_scale(fmaxf(fmaxf(s_max[0][2], s_max[0][3]), fmaxf(s_max[0][6], s_max[0][7])));
            if (is_q) {
                char* hi = I + 2 * kTileBytes;
                put_parts(hi, PARTS > 1 ? hi + kTileBytes : nullptr, i, j0 / 8, s, scale_p);
                put_parts(hi, PARTS > 1 ? hi + kTileBytes : nullptr, i, j0 / 8 + 2, s + 16, scale_p);
            }
            invert(A, M);
            {
                const int i = tid >> 2, j0 = (tid & 3) * 16;
                float x[16], most = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(M + i * LDA + j0 + e);
                    x[e] = j0 + e <= i ? v.x : 0.0f;
                    x[e + 1] = j0 + e + 1 <= i ? v.y : 0.0f;
                    x[e + 2] = j0 + e + 2 <= i ? v.z : 0.0f;
                    x[e + 3] = j0 + e + 3 <= i ? v.w : 0.0f;
                    most = fmaxf(most, fmaxf(fmaxf(fabsf(x[e]), fabsf(x[e + 1])), fmaxf(fabsf(x[e + 2]), fabsf(x[e + 3]))));
                }
                most = warp_max(most);
                if (lane == 0) s_max[1][warp] = most;
                __syncthreads();
                const float scale_m = la::f16_scale(max8(s_max[1]));
                put_parts(I, I + kTileBytes, i, j0 / 8, x, scale_m);
                if (tid == 0) {
                    head->by = s_by[hl].by;
                    head->weak = s_by[hl].weak;
                    head->inv_k = 1.0f / scale_k;
                    head->inv_q = 1.0f / scale_q;
                    head->inv_m = 1.0f / scale_m;
                    head->inv_p = 1.0f / scale_p;
                }
            }
            fence_proxy_async_smem();
            __syncthreads();
            if (tid == 0) {
                la::bulk_store(w.images + ((b * a.H + h) * w.chunks + chunk) * image_bytes(PARTS), I, image_bytes(PARTS));
                la::bulk_commit();
                if (h + 1 < h_hi) la::bulk_wait_read();
            }
        }
    }
    if (tid == 0) la::bulk_wait_all();
    uint64_t* const bars[2] = {&s_ld, &s_mma};
    la::end_block(&s_fail, w.status, bars, tm, 64);
}

template <typename T, int NB, int PARTS> cudaError_t prep_go(const PrepArgs& w, cudaStream_t st) {
    constexpr int bytes = PrepSmem<NB, PARTS>::total;
    const cudaError_t e = la::allow_smem<k_prep<T, NB, PARTS>>(bytes);
    if (e != cudaSuccess) return e;
    k_prep<T, NB, PARTS><<<(unsigned)(w.a.Bsz * w.chunks * w.a.G * w.splits), 256, bytes, st>>>(w);
    return cudaGetLastError();
}
template <typename T, int NB> cudaError_t prep_parts(const PrepArgs& w, int parts, cudaStream_t st) {
    return parts == 1 ? prep_go<T, NB, 1>(w, st) : prep_go<T, NB, 2>(w, st);
}

}  // namespace

cudaError_t launch_prep(const PrepArgs& w, int parts, cudaStream_t st) {
    if (w.a.dtype == 1) return w.a.N <= 64 ? prep_parts<__half, 1>(w, parts, st) : prep_parts<__half, 2>(w, parts, st);
    return w.a.N <= 64 ? prep_parts<bf16, 1>(w, parts, st) : prep_parts<bf16, 2>(w, parts, st);
}

}  // namespace gdr
}  // namespace ss
