// Linear attention, one token per sequence, in place on a pool of states.
//
// state <- e^g state + k v^T, y = scale q state: five operations per state
// element that is read and written once (8 bytes), so the kernel is bound by
// HBM.  A block takes all N rows of LPR * VEC value channels of one (row, head)
// and has every load of its state in flight before it touches q and k.
// Measured: 256 rows x 80 heads of 128 x 64: 195 us, 6.9 TB/s (copying takes 198); one
// row of 24 heads: 2.9 us on the GPU, 15 from Python.
#include "la_dev.cuh"

namespace ss {
namespace la {
namespace {

template <int VEC> struct F;
template <> struct F<4> { using T = float4; };
template <> struct F<1> { using T = float; };

// (wide tiles: five blocks an SM, at 96 registers; the narrow ones of small calls are left alone)
template <typename T, int VEC, int LPR> __global__ void __launch_bounds__(128, LPR == 16 ? 5 : 0) k_step(StepArgs s) {
    constexpr int RP = 128 / LPR;  // state rows the block touches at once
    constexpr int NI = kMaxN / RP;
    constexpr int PT = LPR * VEC;
    __shared__ float s_q[kMaxN], s_k[kMaxN];
    __shared__ float s_y[RP][PT + 1];
    const int tid = threadIdx.x, l = tid % LPR, row = tid / LPR;
    const int64_t ptiles = (s.P + PT - 1) / PT;
    int64_t id = blockIdx.x;
    const int64_t p = (id % ptiles) * PT + l * VEC;
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
    if (tid < s.N) {
        s_q[tid] = ldf(static_cast<const T*>(s.q) + b * s.q_batch + hq * s.N + tid);
        s_k[tid] = ldf(static_cast<const T*>(s.k) + b * s.k_batch + hq * s.N + tid);
    }
    float v[VEC], acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; e++) {
        v[e] = mine ? ldf(static_cast<const T*>(s.v) + b * s.v_batch + h * s.P + p + e) : 0.0f;
        acc[e] = 0.0f;
    }
    const Decay a = decay_of(clamp_g(s.g_per_head ? s.g[h] : s.g[b * s.H + h]));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int n = row + i * RP;
        if (mine && n < s.N) {
            const float kn = s_k[n], qn = s_q[n];
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                x[i].f[e] = fmaf(kn, v[e], decayed(a, x[i].f[e]));
                acc[e] = fmaf(qn, x[i].f[e], acc[e]);
            }
            *reinterpret_cast<FV*>(at + (int64_t)n * s.P) = x[i].v;
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; e++) s_y[row][l * VEC + e] = acc[e];
    __syncthreads();
    const int64_t pt = p - l * VEC;
    for (int c = tid; c < PT; c += 128)
        if (pt + c < s.P) {
            float t = 0.0f;
#pragma unroll 8
            for (int r = 0; r < RP; r++) t += s_y[r][c];
            st(y + pt + c, on ? s.scale * t : 0.0f);
        }
}

template <typename T> cudaError_t step_io(const StepArgs& s, cudaStream_t st) {
    const int64_t BH = s.Bsz * s.H;
    auto blocks = [&](int64_t pt) { return (unsigned)(BH * ceil_div(s.P, pt)); };
    // rows of the state must be whole float4s (the pool itself is 16-byte aligned)
    if (s.P % 4 != 0) k_step<T, 1, 32><<<blocks(32), 128, 0, st>>>(s);
    // fewer blocks than SMs: narrower column tiles spread them over more (24 heads of
    // 128 x 64: 2.9 against 3.3 us; with 384 it would be 5.5 against 5.0)
    else if (BH * ceil_div(s.P, 64) < kSms) k_step<T, 4, 4><<<blocks(16), 128, 0, st>>>(s);
    else k_step<T, 4, 16><<<blocks(64), 128, 0, st>>>(s);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_step(const StepArgs& s, cudaStream_t st) {
    if (s.dtype == 0) return step_io<float>(s, st);
    if (s.dtype == 1) return step_io<__half>(s, st);
    return step_io<__nv_bfloat16>(s, st);
}

}  // namespace la
}  // namespace ss
