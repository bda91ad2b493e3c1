// The gradient of the causal depthwise conv (+ SiLU) for sm_100a, in scan order t:
//   pre_t  = bias + sum_lag w[lag] x_{t-lag}           (recomputed)
//   dpre_t = dout_t silu'(pre_t)                       (dout_t without the SiLU)
//   dx_s   = sum_lag w[lag] dpre_{s+lag},   dw[lag] = sum_t dpre_t x_{t-lag},   db = sum_t dpre_t
// lag = 0 .. W-1 (w here by lag, w[W-1-k] of the taps). Reads x and dout once, writes dx
// once. Along a row a thread takes 16 steps and recomputes the 3 steps behind them, whose dpre
// reach back into its own (8 steps: 72 us against 60 at B8 D1536 L2048 bf16, where HBM needs
// 23: the issue slots bind, 48 instructions an element); channel-last a thread walks a run of 4
// channels down a chunk of 64 steps with the last 3 steps in registers, 4 steps' loads issued
// together (32768 x 1536: 187 us, HBM 61). dw and db are summed per CTA into a partial row
// each, and over the rows by conv_reduce_kernel: no atomics.
#pragma once

#include "scan_bwd_kernel.cuh"

namespace ssm {

constexpr int kConvRun = 16;                                   // steps per thread along a row
constexpr int kConvRowThreads = 128;
constexpr int kConvRowChunk = kConvRun * kConvRowThreads;      // steps per CTA along a row
constexpr int kConvClChunk = 64;                               // steps per thread, channel-last
constexpr int kConvClRun = 4;                                  // channels per thread
constexpr int kConvClAhead = 4;                                // steps whose loads are issued together

// d silu(v) / dv (sigmoidf_ says how exactly)
__device__ __forceinline__ float dsilu(float v) {
    const float s = sigmoidf_(v);
    return s * fmaf(v, 1.f - s, 1.f);
}

template <typename T>
__device__ __forceinline__ float conv_hist(const ConvBwdParams& p, int b, int d, int t) {
    // x at scan position t in [-(W-1), 0)
    return p.hist && t >= -(p.width - 1)
               ? Elem<T>::to_f(static_cast<const T*>(
                     p.hist)[((int64_t)b * p.dim + d) * (p.width - 1) + (p.width - 1 + t)])
               : 0.f;
}

// R elements from p on in the run's direction (rev: towards lower positions), aligned.
template <typename T, int R>
__device__ __forceinline__ void take_dense(const T* p, bool rev, float (&f)[R]) {
    take_run<T, R>(rev ? p - (R - 1) : p, rev, f);
}

template <typename T, bool Q8>
__global__ void __launch_bounds__(kConvRowThreads, 6) conv_bwd_row_kernel(const ConvBwdParams p) {
    constexpr int R = kConvRun;
    using X = std::conditional_t<Q8, int8_t, T>;
    const int L = p.seqlen, dir = p.reverse ? -1 : 1;
    const int64_t rowid = (int64_t)blockIdx.z * 65535 + blockIdx.y;
    if (rowid >= (int64_t)p.batch * p.dim) return;             // below 2^31: a 32-bit division
    const int b = (int)((uint32_t)rowid / (uint32_t)p.dim), d = (int)((uint32_t)rowid % (uint32_t)p.dim);
    const int t0 = blockIdx.x * kConvRowChunk + threadIdx.x * R;
    float w[4];                                                // by lag
#pragma unroll
    for (int lag = 0; lag < 4; ++lag)
        w[lag] = lag < p.width ? p.w[(int64_t)d * p.width + p.width - 1 - lag] : 0.f;
    const float bias = p.bias ? p.bias[d] : 0.f;
    float sw[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
    if (t0 < L) {
        // x[t0 - 3 .. t0 + R + 2], dpre[t0 .. t0 + R + 2]
        float x[R + 6], dp[R + 3];
        const bool rev = p.reverse;
        const int pos0 = rev ? L - 1 - t0 : t0;
        const X* xr = static_cast<const X*>(p.x.p) + (int64_t)b * p.x.s.b + (int64_t)d * p.x.s.c;
        // codes to values: n of them from position ps on in the run's direction, of one block
        auto scaled = [&](float* v, int n, int ps) {
            if constexpr (Q8) {
                const float sc = p.x.scale[(int64_t)b * p.x.ss.b + (int64_t)d * p.x.ss.c + ps / kBlock8];
                for (int i = 0; i < n; ++i) v[i] *= sc;
            }
        };
        const int64_t orow = (int64_t)b * p.sdo.b + (int64_t)d * p.sdo.c;
        if (p.vec && t0 + R <= L) {
            // a whole run of an aligned row: the run, 4 steps before it and 4 behind it
            float run[R], near[4];
            take_dense<X, R>(xr + pos0, rev, run);
            scaled(run, R, pos0);
#pragma unroll
            for (int i = 0; i < R; ++i) x[3 + i] = run[i];
            // (at a row's ends some other 4 of the row in their place, not used: no branch comes
            // between the loads)
            const bool more = t0 + R < L;
            const int before = t0 > 0 ? pos0 - dir * 4 : pos0, after = more ? pos0 + dir * R : pos0;
            take_dense<X, 4>(xr + before, rev, near);
            scaled(near, 4, before);
#pragma unroll
            for (int i = 0; i < 3; ++i) x[i] = near[i + 1];
            take_dense<X, 4>(xr + after, rev, near);
            scaled(near, 4, after);
#pragma unroll
            for (int i = 0; i < 3; ++i) x[R + 3 + i] = more ? near[i] : 0.f;
            if (p.dout32) {
                const float* o = static_cast<const float*>(p.dout) + orow;
                take_dense<float, R>(o + pos0, rev, run);
                take_dense<float, 4>(o + after, rev, near);
            } else {
                const T* o = static_cast<const T*>(p.dout) + orow;
                take_dense<T, R>(o + pos0, rev, run);
                take_dense<T, 4>(o + after, rev, near);
            }
            if (!more)
#pragma unroll
                for (int i = 0; i < 4; ++i) near[i] = 0.f;
            if (t0 == 0)
#pragma unroll
                for (int i = 0; i < 3; ++i) x[i] = conv_hist<T>(p, b, d, i - 3);
#pragma unroll
            for (int i = 0; i < R + 3; ++i) dp[i] = i < R ? run[i < R ? i : 0] : near[i < R ? 0 : i - R];
        } else {
#pragma unroll
            for (int i = 0; i < R + 6; ++i) {
                const int t = t0 - 3 + i;
                x[i] = t < 0 ? conv_hist<T>(p, b, d, t) : t < L ? load_act<T>(p.x, b, d, rev ? L - 1 - t : t) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < R + 3; ++i) {
                const int64_t o = orow + (int64_t)(pos0 + dir * i) * p.sdo.p;
                dp[i] = t0 + i >= L ? 0.f
                        : p.dout32  ? static_cast<const float*>(p.dout)[o]
                                    : Elem<T>::to_f(static_cast<const T*>(p.dout)[o]);
            }
        }
        float dx[R + 3];                                       // dx[t0 - 3 .. t0 + R - 1]
#pragma unroll
        for (int i = 0; i < R + 3; ++i) dx[i] = 0.f;
        // cut: only the taps within the conv's width and the sequence (an absent tap is no
        // product with 0, which a NaN or an infinity would pass)
        auto steps = [&](auto cut) {
#pragma unroll
            for (int i = 0; i < R + 3; ++i) {
                const int sn = decltype(cut)::value ? min(p.since && t0 + i < L ? p.since[t0 + i] : 4, p.width - 1) : 4;
                if (p.silu) {
                    float pre = bias;
#pragma unroll
                    for (int lag = 0; lag < 4; ++lag)
                        if (lag <= sn) pre = fmaf(w[lag], x[3 + i - lag], pre);
                    dp[i] *= dsilu(pre);
                }
#pragma unroll
                for (int lag = 0; lag < 4; ++lag)
                    if (lag <= sn) {
                        if (i - lag < R)
                            dx[i - lag < R ? 3 + i - lag : 0] = fmaf(w[lag], dp[i], dx[i - lag < R ? 3 + i - lag : 0]);
                        if (i < R) sw[lag] = fmaf(dp[i], x[3 + i - lag], sw[lag]);
                    }
                if (i < R) sw[4] += dp[i];
            }
        };
        if (p.since || p.width < 4) steps(std::true_type{});
        else steps(std::false_type{});
        float out[R];
#pragma unroll
        for (int i = 0; i < R; ++i) out[i] = dx[3 + i];
        T* o = static_cast<T*>(p.dx) + (int64_t)b * p.sdx.b + (int64_t)d * p.sdx.c + pos0;
        put_run<T, R>(rev ? o - (R - 1) : o, rev, p.vec, min(R, L - t0), out);
        if (t0 == 0 && p.dhist)
#pragma unroll
            for (int m = 0; m < 3; ++m)                        // positions -3 .. -1
                if (m >= 4 - p.width)
                    static_cast<T*>(p.dhist)[rowid * (p.width - 1) + (p.width - 4 + m)] =
                        Elem<T>::from_f(dx[m]);
    }
    __shared__ __align__(16) float red[5][kConvRowThreads];
#pragma unroll
    for (int k = 0; k < 5; ++k) red[k][threadIdx.x] = sw[k];
    __syncthreads();
    static_assert(kConvRowThreads == 128, "a warp's lanes take 4 threads' sums each");
    for (int k = threadIdx.x / 32; k < 5; k += kConvRowThreads / 32) {
        const float4 q = reinterpret_cast<const float4*>(red[k])[threadIdx.x % 32];
        float v = (q.x + q.y) + (q.z + q.w);
#pragma unroll
        for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (threadIdx.x % 32 == 0) p.part[(((int64_t)b * p.chunks + blockIdx.x) * p.dim + d) * 5 + k] = v;
    }
}

// The first hi of E values at p, the others 0.
template <typename Q, int E>
__device__ __forceinline__ void take_some(const Q* p, int hi, float (&f)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
        f[i] = 0.f;
        if (i < hi) {
            if constexpr (sizeof(Q) == 1) f[i] = (float)p[i];
            else f[i] = Elem<Q>::to_f(p[i]);
        }
    }
}

// Channel-last: only the scan's gradient calls it, with dout in fp32 (dout32).
template <typename T, bool Q8>
__global__ void __launch_bounds__(128) conv_bwd_cl_kernel(const ConvBwdParams p) {
    constexpr int E = kConvClRun, U = kConvClAhead;
    using X = std::conditional_t<Q8, int8_t, T>;
    const int L = p.seqlen;
    // groups of channels times chunks of steps along x: both may pass 65535
    const int groups = (p.dim + 128 * E - 1) / (128 * E);
    const int chunk = blockIdx.x / groups, b = blockIdx.y;
    const int d = ((blockIdx.x - chunk * groups) * 128 + threadIdx.x) * E;
    if (d >= p.dim) return;
    const int hi = min(E, p.dim - d);
    const int tb = chunk * p.chunk_len, te = min(L, tb + p.chunk_len);
    float w[4][E], bias[E], sw[5][E], xw[4][E], acc[4][E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
#pragma unroll
        for (int lag = 0; lag < 4; ++lag) {
            w[lag][i] = i < hi && lag < p.width ? p.w[(int64_t)(d + i) * p.width + p.width - 1 - lag] : 0.f;
            sw[lag][i] = acc[lag][i] = 0.f;
        }
        sw[4][i] = 0.f;
        bias[i] = i < hi && p.bias ? p.bias[d + i] : 0.f;
        xw[3][i] = 0.f;
    }
    auto pos = [&](int t) { return p.reverse ? L - 1 - t : t; };
    const X* xb = static_cast<const X*>(p.x.p) + (int64_t)b * p.x.s.b + d;
    const float* yb = static_cast<const float*>(p.dout) + (int64_t)b * p.sdo.b + d;
    auto scaled = [&](int t, float (&v)[E]) {                  // codes to values
        if constexpr (Q8)
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (i < hi)
                    v[i] *= p.x.scale[(int64_t)b * p.x.ss.b + (int64_t)(pos(t) / kBlock8) * p.x.ss.p + d + i];
    };
    // xw[lag] holds x_{t-lag}; before the first step x_{tb-1-lag}
#pragma unroll
    for (int lag = 0; lag < 3; ++lag) {
        const int t = tb - 1 - lag;
        if (t >= 0) {
            take_some<X, E>(xb + (int64_t)pos(t) * p.x.s.p, hi, xw[lag]);
            scaled(t, xw[lag]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) xw[lag][i] = i < hi ? conv_hist<T>(p, b, d + i, t) : 0.f;
        }
    }
    const bool whole = p.vec && hi == E;
    for (int tu = tb; tu < te + 3; tu += U) {
        float x[U][E], dp[U][E];
        int sn[U];
        if (whole) {                                           // every load before the first use
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int64_t ps = pos(min(tu + k, L - 1));    // past the end: the last step, dropped below
                take_run<X, E>(xb + ps * p.x.s.p, false, x[k]);
                take_run<float, E>(yb + ps * p.sdo.p, false, dp[k]);
            }
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (tu + k >= L)
#pragma unroll
                    for (int i = 0; i < E; ++i) x[k][i] = dp[k][i] = 0.f;
        } else {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int n = tu + k < L ? hi : 0;
                const int64_t ps = n ? pos(tu + k) : 0;
                take_some<X, E>(xb + ps * p.x.s.p, n, x[k]);
                take_some<float, E>(yb + ps * p.sdo.p, n, dp[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k)                            // the furthest tap that is not cut
            sn[k] = min(p.since ? p.since[min(tu + k, L - 1)] : 4, p.width - 1);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int t = tu + k;
            if (t >= te + 3) break;
            if (t < L) scaled(t, x[k]);
            float out[E];
            auto step = [&](auto within) {                     // all 4 taps are there, within the sequence
                constexpr bool all = decltype(within)::value;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    xw[3][i] = xw[2][i];
                    xw[2][i] = xw[1][i];
                    xw[1][i] = xw[0][i];
                    xw[0][i] = x[k][i];
                    acc[3][i] = acc[2][i];                     // acc[lag]: dx_{t-lag} so far
                    acc[2][i] = acc[1][i];
                    acc[1][i] = acc[0][i];
                    acc[0][i] = 0.f;
                    float g = dp[k][i];
                    if (p.silu) {
                        float pre = bias[i];
#pragma unroll
                        for (int lag = 0; lag < 4; ++lag)
                            if (all || lag <= sn[k]) pre = fmaf(w[lag][i], xw[lag][i], pre);
                        g *= dsilu(pre);
                    }
#pragma unroll
                    for (int lag = 0; lag < 4; ++lag)
                        if (all || lag <= sn[k]) acc[lag][i] = fmaf(w[lag][i], g, acc[lag][i]);
                    const float gs = t < te ? g : 0.f;         // the halo's steps are another chunk's
#pragma unroll
                    for (int lag = 0; lag < 4; ++lag)
                        if (all || lag <= sn[k]) sw[lag][i] = fmaf(gs, xw[lag][i], sw[lag][i]);
                    sw[4][i] += gs;
                    out[i] = acc[3][i];
                }
            };
            if (sn[k] >= 3) step(std::true_type{});
            else step(std::false_type{});
            const int s = t - 3;                               // dx_s is complete
            if (s >= tb) {
                put_run<T, E>(static_cast<T*>(p.dx) + (int64_t)b * p.sdx.b + d + (int64_t)pos(s) * p.sdx.p,
                              false, p.vec, hi, out);
            } else if (chunk == 0 && p.dhist && s >= -(p.width - 1)) {
#pragma unroll
                for (int i = 0; i < E; ++i)
                    if (i < hi)
                        static_cast<T*>(p.dhist)[((int64_t)b * p.dim + d + i) * (p.width - 1) +
                                                 (p.width - 1 + s)] = Elem<T>::from_f(out[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < hi)
#pragma unroll
            for (int k = 0; k < 5; ++k)
                p.part[(((int64_t)b * p.chunks + chunk) * p.dim + d + i) * 5 + k] = sw[k][i];
}

// dw (dim, width), dbias (dim) from the partial rows (rows, dim, 5: by lag, then bias). A CTA
// takes 32 columns; its 8 warps take the rows in turn and meet in shared memory.
__global__ void __launch_bounds__(256) conv_reduce_kernel(const ConvReduceParams p) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t idx = (int64_t)blockIdx.x * 32 + lane;
    LongSum sum;
    if (idx < (int64_t)p.dim * 5) {
#pragma unroll 8
        for (int64_t r = warp; r < p.rows; r += 8) sum.add(p.part[r * p.dim * 5 + idx]);
    }
    float v = sum.get();
    red[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || idx >= (int64_t)p.dim * 5) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) v += red[k][lane];
    const int d = (int)(idx / 5), k = (int)(idx % 5);
    if (k < 4) {
        if (p.dw && k < p.width) p.dw[(int64_t)d * p.width + p.width - 1 - k] = v;
    } else if (p.dbias) {
        p.dbias[d] = v;
    }
}

}  // namespace ssm
