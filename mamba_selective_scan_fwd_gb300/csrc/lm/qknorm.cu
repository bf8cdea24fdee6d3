// Norm of each head's channels of q and k with the rotation by position, forward
// and backward.
//
//   n = x r w,  r = 1 / sqrt(mean(x^2) + eps) (or of the sum);  out = turn(n)
//   d = turn back(dout);  dw = sum d x r;  dx = r (d w - x r m (d w . x r)),  m = 1 / N (or 1)
// Both directions are bound by HBM: a row (one head of one token) is read once into
// the registers of a few lanes and written once.  A lane holds two runs of V channels,
// chosen so that the channels that turn together are its own: i and i + pairs, or
// neighbours.  Statistics are f32.  A tile of tokens shares one table of angles in shared
// memory, used by all heads; position * frequency is reduced to a fraction of a turn by a
// 64-bit product (the frequency as a fraction of 2^64 turns a token).  What is left of the
// angle is good to 2^-26 turns, its own f32, and 2^-52 of the turns made, the frequency's
// quotient by 2 pi in 53 bits: 2^-23 at a radian a token and 2^31 tokens.
//
// A row's loads are on their way while the row before it is worked on, over the tiles' ends too: the next
// tile's tables are made first.  Measured: 4 x 4096 tokens, 16 + 16 heads of 128, 64 channels turned: 48 us, copying 40
// (tables and loads begun anew at each tile: 55); backward of half of it 41 + 3, three streams at the copy rate 30
// (50 + 6): 123 registers let two blocks of 256 fit an SM, and the same with 64 registers and runs of half the width
// takes 57.  All 128 channels turned, 2 x 4096 tokens: 29 us for 20 of copying; few heads a token: bound by the angles.  f32, 4 x 4096
// tokens: 89 us a call for 79 of copying, the gradient 134 for 119.
#include "../simd.cuh"
#include "gdr_dev.cuh"
#include "ss_gdr.h"

namespace ss {
namespace gdr {
namespace {

constexpr int kThreads = 256;
// A frequency that is not finite.  (No fraction is this: those of 2^62 and more come from 53 bits and are multiples of 2^10.)
constexpr uint64_t kNoAngle = (1ull << 62) + 1;
constexpr int kTable = 1024;  // angles a tile of tokens may need (8 KB)
constexpr int kTile = 128;    // tokens of a tile at most

template <typename T, int V> struct Run {  // V values moved at once
    using M = typename std::conditional<sizeof(T) * V == 16, uint4, typename std::conditional<sizeof(T) * V == 8, uint2, T>::type>::type;
};
template <typename T, int V> __device__ __forceinline__ void widen(const typename Run<T, V>::M& m, float (&f)[V]) {
    union {
        typename Run<T, V>::M m;
        T t[V];
    } u;
    u.m = m;
#pragma unroll
    for (int e = 0; e < V; e++) f[e] = ldf(&u.t[e]);
}
template <typename T, int V> __device__ __forceinline__ void put(T* p, const float (&f)[V]) {
    union {
        typename Run<T, V>::M m;
        T t[V];
    } u;
#pragma unroll
    for (int e = 0; e < V; e++) st(&u.t[e], f[e]);
    *reinterpret_cast<typename Run<T, V>::M*>(p) = u.m;
}

// LPR lanes a row, SPT pairs of runs a lane.  Block (x, side): tiles of `tile` tokens of
// q (side 0) or k.
template <typename T, int V, int LPR, int SPT, bool BWD>
__global__ void __launch_bounds__(kThreads) k_qknorm(NormArgs a, int64_t tile, int64_t blocks_q) {
    constexpr int RPB = kThreads / LPR;  // rows at once
    // three tiles' tables: of the one in work, of the next (its rows are fetched before this one's end), and of the one
    // before, which slower warps may still read.  One barrier a tile.
    __shared__ float2 s_turn[3][kTable];
    __shared__ int64_t s_at[3][BWD ? 2 : 1][kTile];  // where each token of the tile begins in x (and in d)
    __shared__ uint64_t s_freq[la::kMaxN];
    __shared__ float s_dw[BWD ? 2 * V * SPT * kThreads : 1];
    const int sd = blockIdx.x >= blocks_q;
    const NormSide& z = a.side[sd];
    const int64_t block = blockIdx.x - (sd ? blocks_q : 0), blocks = sd ? gridDim.x - blocks_q : blocks_q;
    const int tid = threadIdx.x, sub = tid % LPR, slot = tid / LPR;
    const int N = (int)a.N, pairs = (int)a.pairs, heads = (int)z.heads;
    const bool l2 = a.flags & SS_QKNORM_L2, inter = a.flags & SS_QKNORM_INTERLEAVED;
    const int64_t tokens = a.Bsz * a.L;
    for (int i = tid; i < pairs; i += kThreads) {
        const double t = (double)a.freqs[i] * 0.15915494309189533577;  // turns a token
        double f = t - rint(t);  // exact: the distance to the whole turn below would round tiny negative ones to one
        if (f >= 0.5) f -= 1.0;  // -1/2 .. 1/2, what 64 bits hold with their sign
        s_freq[i] = isfinite(t) ? (uint64_t)(int64_t)(f * 18446744073709551616.0) : kNoAngle;
    }
    // the lane's runs: channels ia .. + V - 1 and ib ..; turned: the angles i0 .. (of the row's table), V or V / 2 a run
    int ia[SPT], ib[SPT], i0[SPT];
    bool on[SPT], onb[SPT], turned[SPT];
    float w[SPT][2][V], dw[SPT][2][V];
#pragma unroll
    for (int s = 0; s < SPT; s++) {
        const int at = (sub + LPR * s) * V;  // of pairs of channels
        turned[s] = at < pairs;
        const bool halves = turned[s] && !inter;
        ia[s] = halves ? at : 2 * at;
        ib[s] = halves ? at + pairs : 2 * at + V;
        i0[s] = at;
        on[s] = ia[s] < N;
        onb[s] = ib[s] < N;
#pragma unroll
        for (int e = 0; e < V; e++) {
            w[s][0][e] = z.weight && on[s] ? z.weight[ia[s] + e] : 1.0f;
            w[s][1][e] = z.weight && onb[s] ? z.weight[ib[s] + e] : 1.0f;
            dw[s][0][e] = dw[s][1][e] = 0.0f;
        }
    }
    // one run's turn by angles: (A, B) as halves or A and B each of neighbours; back: by the opposite angle
    auto turn = [&](float (&x)[2][V], const float2* cs, bool halves, float sign) {
        if (halves || V == 1) {
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float2 t = cs[e];
                const float A = x[0][e], B = x[1][e], sn = sign * t.y;
                x[0][e] = A * t.x - B * sn;
                x[1][e] = B * t.x + A * sn;
            }
        } else {
#pragma unroll
            for (int r = 0; r < 2; r++)
#pragma unroll
                for (int e = 0; e + 1 < V; e += 2) {
                    const float2 t = cs[(r * V + e) / 2];
                    const float A = x[r][e], B = x[r][e + (V > 1)], sn = sign * t.y;
                    x[r][e] = A * t.x - B * sn;
                    x[r][e + (V > 1)] = B * t.x + A * sn;
                }
        }
    };
    const float inv = l2 ? 1.0f : 1.0f / (float)N;
    using M = typename Run<T, V>::M;
    struct Raw {
        M x[SPT][2], d[BWD ? SPT : 1][2];
    };
    auto tables = [&](int at, int64_t t0) {
        const int nt = (int)min(tile, tokens - t0);
        const int64_t b0 = t0 / a.L, first = t0 - b0 * a.L;  // (divisions of 64 bits: once a tile)
        for (int i = tid; i < nt; i += kThreads) {
            const int64_t over = first + i >= a.L ? (a.L >= tile ? 1 : (first + i) / a.L) : 0;
            const int64_t b = b0 + over, tb = first + i - over * a.L;
            s_at[at][0][i] = b * z.x.batch + tb * z.x.token;
            if (BWD) s_at[at][BWD][i] = b * z.d.batch + tb * z.d.token;
        }
        for (int i = tid; i < nt * pairs; i += kThreads) {
            const int tl = i / pairs;
            int64_t pos = first + tl;
            if (a.positions) pos = a.positions[t0 + tl];
            else if (pos >= a.L) pos = a.L >= tile ? pos - a.L : pos % a.L;
            const uint64_t f = s_freq[i - tl * pairs];
            const float part = (float)(int32_t)(((uint64_t)pos * f + 0x80000000ull) >> 32) * 4.656612873077393e-10f;  // half turns
            float sn, cs;
            sincospif(part, &sn, &cs);
            s_turn[at][i] = f == kNoAngle ? make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff)) : make_float2(cs, sn);
        }
    };
    auto fetch = [&](int at, int tl, int h, bool have, Raw& raw) {  // a row's runs on their way
        const T* xp = static_cast<const T*>(z.x.p) + (have ? s_at[at][0][tl] + (int64_t)h * N : 0);
        const T* dp = BWD ? static_cast<const T*>(z.d.p) + (have ? s_at[at][BWD][tl] + (int64_t)h * N : 0) : nullptr;
#pragma unroll
        for (int s = 0; s < SPT; s++) {
            raw.x[s][0] = raw.x[s][1] = M{};
            if (have && on[s]) raw.x[s][0] = *reinterpret_cast<const M*>(xp + ia[s]);
            if (have && onb[s]) raw.x[s][1] = *reinterpret_cast<const M*>(xp + ib[s]);
            if (BWD) {
                raw.d[BWD ? s : 0][0] = raw.d[BWD ? s : 0][1] = M{};
                if (have && on[s]) raw.d[BWD ? s : 0][0] = *reinterpret_cast<const M*>(dp + ia[s]);
                if (have && onb[s]) raw.d[BWD ? s : 0][1] = *reinterpret_cast<const M*>(dp + ib[s]);
            }
        }
    };
    const int tl0 = slot / heads, h0 = slot - tl0 * heads, dt = RPB / heads, dh = RPB - dt * heads;
    Raw next;
    int at = 0;
    __syncthreads();  // the frequencies
    if (block * tile < tokens) {
        tables(0, block * tile);
        __syncthreads();
        fetch(0, tl0, h0, tl0 < min(tile, tokens - block * tile), next);
    }
    for (int64_t t0 = block * tile; t0 < tokens; t0 += blocks * tile) {
        const int nt = (int)min(tile, tokens - t0), rows = nt * heads;
        const int64_t t1 = t0 + blocks * tile;
        const int nt1 = (int)max((int64_t)0, min(tile, tokens - t1)), at1 = at == 2 ? 0 : at + 1;
        if (nt1 > 0) tables(at1, t1);
        __syncthreads();
        int tl = tl0, h = h0;
        for (int r0 = 0; r0 < rows; r0 += RPB) {
            const bool have = tl < nt;
            const int64_t t = t0 + tl;
            float x[SPT][2][V], d[SPT][2][V];
            float sum = 0.0f;
#pragma unroll
            for (int s = 0; s < SPT; s++)
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    widen<T, V>(next.x[s][c], x[s][c]);
                    if (BWD) widen<T, V>(next.d[BWD ? s : 0][c], d[s][c]);
                }
            const int now = tl, head = h;
            h += dh;
            tl += dt;
            if (h >= heads) {
                h -= heads;
                tl++;
            }
            if (r0 + RPB < rows) fetch(at, tl, h, tl < nt, next);
            else fetch(at1, tl0, h0, tl0 < nt1, next);
#pragma unroll
            for (int s = 0; s < SPT; s++)
#pragma unroll
                for (int e = 0; e < V; e++) sum = fmaf(x[s][0][e], x[s][0][e], fmaf(x[s][1][e], x[s][1][e], sum));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            const float rs = rsqrtf(fmaf(sum, inv, a.eps));
            const float2* cs = s_turn[at] + (have ? now * pairs : 0);
            T* op = static_cast<T*>(z.out) + (t * heads + head) * N;
            if (!BWD) {
#pragma unroll
                for (int s = 0; s < SPT; s++) {
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        x[s][0][e] *= rs * w[s][0][e];
                        x[s][1][e] *= rs * w[s][1][e];
                    }
                    if (turned[s]) turn(x[s], cs + i0[s], !inter, 1.0f);
                    if (have && on[s]) put<T, V>(op + ia[s], x[s][0]);
                    if (have && onb[s]) put<T, V>(op + ib[s], x[s][1]);
                }
            } else {
                float dot = 0.0f;
#pragma unroll
                for (int s = 0; s < SPT; s++) {
                    if (turned[s]) turn(d[s], cs + i0[s], !inter, -1.0f);
#pragma unroll
                    for (int c = 0; c < 2; c++)
#pragma unroll
                        for (int e = 0; e < V; e++) {
                            x[s][c][e] *= rs;  // x r
                            if (have) dw[s][c][e] = fmaf(d[s][c][e], x[s][c][e], dw[s][c][e]);
                            d[s][c][e] *= w[s][c][e];
                            dot = fmaf(d[s][c][e], x[s][c][e], dot);
                        }
                }
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
                const float m = inv * dot;
#pragma unroll
                for (int s = 0; s < SPT; s++) {
#pragma unroll
                    for (int c = 0; c < 2; c++)
#pragma unroll
                        for (int e = 0; e < V; e++) d[s][c][e] = rs * fmaf(-m, x[s][c][e], d[s][c][e]);
                    if (have && on[s]) put<T, V>(op + ia[s], d[s][0]);
                    if (have && onb[s]) put<T, V>(op + ib[s], d[s][1]);
                }
            }
        }
        at = at1;
    }
    if (BWD && z.dweight) {  // the block's sum over its rows, slots in order
        __syncthreads();
#pragma unroll
        for (int s = 0; s < SPT; s++)
#pragma unroll
            for (int c = 0; c < 2; c++)
#pragma unroll
                for (int e = 0; e < V; e++) s_dw[((s * 2 + c) * V + e) * kThreads + tid] = dw[s][c][e];
        __syncthreads();
        float* part = a.part + (int64_t)blockIdx.x * N;
        for (int i = tid; i < 2 * V * SPT * LPR; i += kThreads) {
            const int lane = i % LPR, e = i / LPR % V, c = i / LPR / V % 2, s = i / LPR / V / 2;
            const int at = (lane + LPR * s) * V;
            const bool halves = at < pairs && !inter;
            const int n = (c ? (halves ? at + pairs : 2 * at + V) : (halves ? at : 2 * at)) + e;
            float x = 0.0f;
            for (int r = 0; r < RPB; r++) x += s_dw[((s * 2 + c) * V + e) * kThreads + r * LPR + lane];
            if (n < N) part[n] = x;
        }
    }
}

// Weights' gradients: the blocks' parts in order.  Block: 32 channels of one side, 32 warps
// taking every 32nd part.
__global__ void __launch_bounds__(1024) k_weights(NormArgs a, int64_t blocks_q, int64_t blocks) {
    __shared__ float s[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sd = blockIdx.y;
    const int64_t n = (int64_t)blockIdx.x * 32 + lane;
    float* out = a.side[sd].dweight;
    if (!out) return;
    float v = 0.0f;
    if (n < a.N)
#pragma unroll 16
        for (int64_t i = (sd ? blocks_q : 0) + warp; i < (sd ? blocks : blocks_q); i += 32) v += a.part[i * a.N + n];
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && n < a.N) {
        float t = 0.0f;
#pragma unroll
        for (int u = 0; u < 32; u++) t += s[u][lane];
        out[n] = t;
    }
}

// Tokens of a tile: about four rounds of rows, angles within the table.
int64_t tile_tokens(int64_t heads, int64_t pairs, int lanes) {
    int64_t t = ceil_div(4 * (kThreads / lanes), heads);
    if (pairs > 0 && t * pairs > kTable) t = kTable / pairs;
    if (t > kTile) t = kTile;
    return t < 1 ? 1 : t;
}

template <typename T, int V, int LPR, int SPT, bool BWD> cudaError_t launch(const NormArgs& a, cudaStream_t st) {
    static const int fit = [] {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_qknorm<T, V, LPR, SPT, BWD>, kThreads, 0) == cudaSuccess && n > 0 ? n : 1;
    }();
    const int64_t tokens = a.Bsz * a.L, hq = a.side[0].heads, hk = a.side[1].heads, per_sm = fit < kNormBlocks ? fit : kNormBlocks;
    const int64_t bq = norm_blocks(tokens, hq, hk, a.N, per_sm), bk = norm_blocks(tokens, hk, hq, a.N, per_sm);
    k_qknorm<T, V, LPR, SPT, BWD><<<(unsigned)(bq + bk), kThreads, 0, st>>>(a, tile_tokens(hq > hk ? hq : hk, a.pairs, LPR), bq);
    if (BWD && (a.side[0].dweight || a.side[1].dweight))
        k_weights<<<dim3((unsigned)ceil_div(a.N, 32), 2), 1024, 0, st>>>(a, bq, bq + bk);
    return cudaGetLastError();
}
template <typename T, int V, int LPR, int SPT> cudaError_t launch(const NormArgs& a, bool bwd, cudaStream_t st) {
    return bwd ? launch<T, V, LPR, SPT, true>(a, st) : launch<T, V, LPR, SPT, false>(a, st);
}

bool runs_of(const NormArgs& a, bool bwd, int64_t v, int64_t esz) {
    if (a.N % (2 * v) != 0 || a.pairs % v != 0) return false;
    auto ok = [&](const void* p, int64_t token, int64_t batch) {
        return reinterpret_cast<uintptr_t>(p) % (v * esz) == 0 && token % v == 0 && batch % v == 0;
    };
    for (const NormSide& s : a.side)
        if (!ok(s.x.p, s.x.token, s.x.batch) || !ok(s.out, 0, 0) || (bwd && !ok(s.d.p, s.d.token, s.d.batch))) return false;
    return true;
}

// lanes: the power of two that holds the row's pairs of runs
template <typename T, int V> cudaError_t launch_runs(const NormArgs& a, bool bwd, cudaStream_t st) {
    const int64_t need = a.N / (2 * V);
    if (need <= 4) return launch<T, V, 4, 1>(a, bwd, st);
    if (need <= 8) return launch<T, V, 8, 1>(a, bwd, st);
    if (need <= 16) return launch<T, V, 16, 1>(a, bwd, st);
    return launch<T, V, 32, 1>(a, bwd, st);
}

// Runs of 16 bytes where everything is aligned, of 8 or single values else: 4 x 4096 tokens, 16 + 16 heads of 128, bf16, 48 us (backward
// 72), 74 (102), 151 (344).
template <typename T> cudaError_t launch_io(const NormArgs& a, bool bwd, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (runs_of(a, bwd, V, sizeof(T))) return launch_runs<T, V>(a, bwd, st);
    if (V == 8 && runs_of(a, bwd, 4, sizeof(T))) return launch_runs<T, 4>(a, bwd, st);
    if (a.N <= 64) return launch<T, 1, 32, 1>(a, bwd, st);
    return launch<T, 1, 32, 4>(a, bwd, st);
}

}  // namespace

int64_t norm_blocks(int64_t tokens, int64_t heads, int64_t others, int64_t N, int64_t per_sm) {
    const int64_t n = ceil_div(tokens * heads * N, 2048), most = per_sm * kSms * heads / (heads + others);
    return n < 1 || most < 1 ? 1 : (n > most ? most : n);
}

cudaError_t launch_qknorm(const NormArgs& a, bool bwd, cudaStream_t st) {
    if (a.dtype == 0) return launch_io<float>(a, bwd, st);
    if (a.dtype == 1) return launch_io<__half>(a, bwd, st);
    return launch_io<__nv_bfloat16>(a, bwd, st);
}

}  // namespace gdr
}  // namespace ss
