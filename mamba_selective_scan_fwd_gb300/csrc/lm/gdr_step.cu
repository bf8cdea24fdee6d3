// Gated delta rule, one token per sequence, in place on a pool of states.
//
//   S' = e^g S + k u^T with u = beta (v - e^g S^T k),   y = scale q S' = scale (e^g S^T q + (q . k) u)
// Both products with the old state are taken in the one pass that reads it, so that
// the new state needs no second sum over its rows.  Seven operations per state
// element that is read and written once (8 bytes): bound by HBM.  A block takes all N
// rows of LPR * VEC value channels of one (row, head) and keeps them in registers
// between the products and the update.
#include "gdr.h"
#include "la_dev.cuh"

namespace ss {
namespace gdr {
namespace {

using la::ldf;

template <int VEC> struct F;
template <> struct F<4> { using T = float4; };
template <> struct F<1> { using T = float; };

template <typename T, int VEC, int LPR, int THREADS = 128>
__global__ void __launch_bounds__(THREADS, VEC == 4 && LPR >= 16 ? 512 / THREADS : 0) k_step(StepArgs s) {
    constexpr int RP = THREADS / LPR;  // state rows the block touches at once
    constexpr int NI = kMaxN / RP;
    constexpr int PT = LPR * VEC;
    __shared__ float s_q[kMaxN], s_k[kMaxN], s_qk[4];
    __shared__ float s_d[2][RP][PT + 1];
    __shared__ float s_u[PT];
    const int tid = threadIdx.x, l = tid % LPR, row = tid / LPR;
    const int64_t ptiles = (s.P + PT - 1) / PT;
    int64_t id = blockIdx.x;
    const int64_t pt = (id % ptiles) * PT, p = pt + l * VEC;
    id /= ptiles;
    const int64_t h = id % s.H, b = id / s.H;
    const int64_t slot = s.slots ? s.slots[b] : b;
    const bool on = slot >= 0 && slot < s.pool;
    T* y = static_cast<T*>(s.y) + (b * s.H + h) * s.P;
    using FV = typename F<VEC>::T;
    union U {
        FV v;
        float f[VEC];
    } x[NI];
    float* at = s.state + (slot * s.H + h) * s.N * s.P + p;
    const bool mine = on && p < s.P;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int n = row + i * RP;
        if (mine && n < s.N) x[i].v = *reinterpret_cast<const FV*>(at + (int64_t)n * s.P);
    }
    const int64_t hq = h / (s.H / s.G);
    float qn = 0.0f, kn = 0.0f;
    if (tid < s.N) {
        qn = ldf(static_cast<const T*>(s.q) + b * s.q_batch + hq * s.N + tid);
        kn = ldf(static_cast<const T*>(s.k) + b * s.k_batch + hq * s.N + tid);
    }
    if (tid < kMaxN) {
        s_q[tid] = qn;
        s_k[tid] = kn;
    }
    float qk = qn * kn;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) qk += __shfl_xor_sync(kFull, qk, o);
    if ((tid & 31) == 0 && tid < kMaxN) s_qk[tid >> 5] = qk;
    const la::Decay a = la::decay_of(s.g ? la::clamp_g(s.g[b * s.H + h]) : 0.0f);
    const float beta = s.beta[b * s.H + h];
    __syncthreads();
    float dk[VEC], dq[VEC];
#pragma unroll
    for (int e = 0; e < VEC; e++) dk[e] = dq[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int n = row + i * RP;
        if (mine && n < s.N) {
            const float kk = s_k[n], qq = s_q[n];
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                x[i].f[e] = la::decayed(a, x[i].f[e]);
                dk[e] = fmaf(kk, x[i].f[e], dk[e]);
                dq[e] = fmaf(qq, x[i].f[e], dq[e]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; e++) {
        s_d[0][row][l * VEC + e] = dk[e];
        s_d[1][row][l * VEC + e] = dq[e];
    }
    __syncthreads();
    for (int c = tid; c < PT; c += THREADS)
        if (pt + c < s.P) {
            float k_s = 0.0f, q_s = 0.0f;
#pragma unroll 8
            for (int r = 0; r < RP; r++) {
                k_s += s_d[0][r][c];
                q_s += s_d[1][r][c];
            }
            const float u = on ? beta * (ldf(static_cast<const T*>(s.v) + b * s.v_batch + h * s.P + pt + c) - k_s) : 0.0f;
            s_u[c] = u;
            st(y + pt + c, on ? s.scale * fmaf((s_qk[0] + s_qk[1]) + (s_qk[2] + s_qk[3]), u, q_s) : 0.0f);
        }
    __syncthreads();
    float u[VEC];
#pragma unroll
    for (int e = 0; e < VEC; e++) u[e] = mine ? s_u[l * VEC + e] : 0.0f;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int n = row + i * RP;
        if (mine && n < s.N) {
#pragma unroll
            for (int e = 0; e < VEC; e++) x[i].f[e] = fmaf(s_k[n], u[e], x[i].f[e]);
            *reinterpret_cast<FV*>(at + (int64_t)n * s.P) = x[i].v;
        }
    }
}

template <typename T> cudaError_t step_io(const StepArgs& s, cudaStream_t st) {
    const int64_t BH = s.Bsz * s.H;
    auto blocks = [&](int64_t pt) { return (unsigned)(BH * ceil_div(s.P, pt)); };
    // rows of the state must be whole float4s (the pool itself is 16-byte aligned)
    if (s.P % 4 != 0) k_step<T, 1, 32><<<blocks(32), 128, 0, st>>>(s);
    // fewer channels a block where there are SMs for them (one row of 32 heads, N = P = 128: 3.6 us, 4.5 with 64)
    else if (BH * ceil_div(s.P, 64) < kSms) k_step<T, 4, 4><<<blocks(16), 128, 0, st>>>(s);
    // 128 channels at once where they cost no idle lanes over 64: whole rows of 512 bytes (256 rows of 32 heads, N = P = 128:
    // 174 us, 184 with 64, 192 with 32; copying 159)
    else if (ceil_div(s.P, 64) % 2 == 1) k_step<T, 4, 16><<<blocks(64), 128, 0, st>>>(s);
    else k_step<T, 4, 32, 256><<<blocks(128), 256, 0, st>>>(s);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_step(const StepArgs& s, cudaStream_t st) {
    if (s.dtype == 0) return step_io<float>(s, st);
    if (s.dtype == 1) return step_io<__half>(s, st);
    return step_io<__nv_bfloat16>(s, st);
}

}  // namespace gdr
}  // namespace ss
