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

template <int NB, int PARTS> struct PrepSmem {
    static constexpr int kq = 0, image = NB * 16384, a = image + image_bytes(PARTS), m = a + C * LDA * 4, total = m + C * LDA * 4;
};

// 16 values as two bf16 parts, in units u0, u0 + 1 of a row of two tiles
__device__ __forceinline__ void put_parts(char* hi, char* lo, int row, int u0, const float (&x)[16]) {
#pragma unroll
    for (int u = 0; u < 2; u++) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = make_float2(x[8 * u + 2 * i], x[8 * u + 2 * i + 1]);
            h[i] = pack2<bf16>(f.x, f.y);
            const float2 r = unpack2<bf16>(h[i]);
            l[i] = pack2<bf16>(f.x - r.x, f.y - r.y);
        }
        *unit(hi, row, u0 + u) = make_uint4(h[0], h[1], h[2], h[3]);
        if (lo) *unit(lo, row, u0 + u) = make_uint4(l[0], l[1], l[2], l[3]);
    }
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
__global__ void __launch_bounds__(256, 2) k_prep(const __grid_constant__ PrepArgs w) {
    extern __shared__ __align__(1024) char sm[];
    using L = PrepSmem<NB, PARTS>;
    __shared__ __align__(8) uint64_t s_ld, s_mma;
    __shared__ uint32_t s_tm, s_fail;
    __shared__ Two s_c[C];
    const Args& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31;
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
    }
    if (tid < 32) la::tmem_alloc(&s_tm, 64);
    __syncthreads();
    la::tc_fence_after();
    const uint32_t tm = s_tm, my = (uint32_t)(tid & 96) << 16;
    if (tid == 0) {
        mbar_expect_tx(&s_ld, NB * 16384);
#pragma unroll
        for (int n = 0; n < NB; n++) {
            la::tma_load_4d(KQ + n * 16384, &w.k, n * 64, (int)gq, (int)t0, (int)b, &s_ld);
            la::tma_load_4d(KQ + n * 16384 + 8192, &w.q, n * 64, (int)gq, (int)t0, (int)b, &s_ld);
        }
        if (la::wait_or_fail(&s_ld, 0, &s_fail)) {
            constexpr uint32_t d = la::mma_desc<T>(128, 64, false, false);
            const uint32_t at = smem_addr(KQ);
#pragma unroll
            for (int s = 0; s < 4 * NB; s++) {
                const uint32_t x = at + (s >> 2) * 16384 + (s & 3) * 32;
                la::mma(tm, la::smem_desc(x), la::smem_desc(x), d, s > 0);
            }
            la::mma_commit(&s_mma);
        }
    }
    __syncwarp();
    bool ok = true;
    for (int64_t h = gq * rep + rep * split / w.splits; h < gq * rep + rep * (split + 1) / w.splits; h++) {
        if (tid < 32) {
            float g[2], x[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int t = 2 * lane + e;
                g[e] = t < nv ? log_decay(a, b, t0 + t, h) : 0.0f;
                x[e] = g[e] * la::kLog2e;
            }
            Two c[2], n[2];
            la::warp_cumsum<2>(x, c);
            la::warp_cumsum<2>(g, n);
            const Two cl = {__shfl_sync(kFull, c[1].h, 31), __shfl_sync(kFull, c[1].l, 31)};
            if (lane == 31) {
                const la::Decay d = la::decay_of(n[1].h + n[1].l);
                head->by = d.by;
                head->weak = d.weak;
            }
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int t = 2 * lane + e;
                s_c[t] = c[e];
                head->up[t] = la::ex2(c[e].h + c[e].l);
                head->down[t] = la::ex2(two_diff(cl, c[e]));
                head->beta[t] = t < nv ? a.beta[(b * a.L + t0 + t) * a.H + h] : 0.0f;
            }
        }
        ok = ok && la::wait_or_fail(&s_mma, 0, &s_fail);
        if (__syncthreads_or(!ok)) break;
        la::tc_fence_after();
        {  // thread: row i of K K^T (warps 0, 1 of a warpgroup) or Q K^T, 32 columns
            const bool is_q = tid & 64;
            const int i = tid & 63, j0 = (tid >> 7) * 32;
            float s[32];
            la::tmem_ld32(tm + my + j0, s);
            const Two ci = s_c[i];
            const float f = is_q ? 1.0f : head->beta[i];
            const bool own = i < nv;
            const int last = is_q ? i : i - 1;
#pragma unroll
            for (int j = 0; j < 32; j++) {
                const int col = j0 + j;
                s[j] = own && col <= last ? f * s[j] * la::ex2(two_diff(ci, s_c[col])) : 0.0f;
            }
            if (is_q) {
                char* hi = I + 2 * kTileBytes;
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    float x[16];
#pragma unroll
                    for (int e = 0; e < 16; e++) x[e] = s[16 * u + e];
                    put_parts(hi, PARTS > 1 ? hi + kTileBytes : nullptr, i, j0 / 8 + 2 * u, x);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<float4*>(A + i * LDA + j0 + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
            }
        }
        __syncthreads();
        invert(A, M);
        {
            const int i = tid >> 2, j0 = (tid & 3) * 16;
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const float4 v = *reinterpret_cast<const float4*>(M + i * LDA + j0 + e);
                x[e] = j0 + e <= i ? v.x : 0.0f;
                x[e + 1] = j0 + e + 1 <= i ? v.y : 0.0f;
                x[e + 2] = j0 + e + 2 <= i ? v.z : 0.0f;
                x[e + 3] = j0 + e + 3 <= i ? v.w : 0.0f;
            }
            put_parts(I, I + kTileBytes, i, j0 / 8, x);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            la::bulk_store(w.images + ((b * a.H + h) * w.chunks + chunk) * image_bytes(PARTS), I, image_bytes(PARTS));
            la::bulk_commit();
            la::bulk_wait_read();
        }
        __syncthreads();
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
