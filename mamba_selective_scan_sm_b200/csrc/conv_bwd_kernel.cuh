// The gradient of the causal depthwise conv (+ SiLU) for sm_100a, in scan order t:
//   pre_t  = bias + sum_lag w[lag] x_{t-lag}           (recomputed)
//   dpre_t = dout_t silu'(pre_t)                       (dout_t without the SiLU)
//   dx_s   = sum_lag w[lag] dpre_{s+lag},   dw[lag] = sum_t dpre_t x_{t-lag},   db = sum_t dpre_t
// lag = 0 .. W-1 (w here by lag, w[W-1-k] of the taps). Reads x and dout once, writes dx
// once: bound by memory. Along a row a thread takes 8 steps and recomputes the 3 steps
// behind them, whose dpre reach back into its own; channel-last a thread walks a run of
// channels down a chunk of steps with the last 3 steps in registers. dw and db are summed
// per CTA into a partial row each, and over the rows by conv_reduce_kernel: no atomics.
#pragma once

#include "scan_bwd_kernel.cuh"

namespace ssm {

constexpr int kConvRun = 8;                                    // steps per thread along a row
constexpr int kConvRowThreads = 128;
constexpr int kConvRowChunk = kConvRun * kConvRowThreads;      // steps per CTA along a row
constexpr int kConvClChunk = 64;                               // steps per thread, channel-last
constexpr int kConvClRun = 4;                                  // channels per thread

// d silu(v) / dv
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

template <typename T>
__global__ void __launch_bounds__(kConvRowThreads) conv_bwd_row_kernel(const ConvBwdParams p) {
    constexpr int R = kConvRun;
    const int L = p.seqlen, dir = p.reverse ? -1 : 1;
    const int64_t rowid = (int64_t)blockIdx.z * 65535 + blockIdx.y;
    if (rowid >= (int64_t)p.batch * p.dim) return;
    const int b = (int)(rowid / p.dim), d = (int)(rowid % p.dim);
    const int t0 = blockIdx.x * kConvRowChunk + threadIdx.x * R;
    float w[4];                                                // by lag
#pragma unroll
    for (int lag = 0; lag < 4; ++lag)
        w[lag] = lag < p.width ? p.w[(int64_t)d * p.width + p.width - 1 - lag] : 0.f;
    const float bias = p.bias ? p.bias[d] : 0.f;
    float sw[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
    if (t0 < L) {
        // x[t0 - 3 .. t0 + 10], dpre[t0 .. t0 + 10]
        float x[R + 6], dp[R + 3], run[R];
        auto pos = [&](int t) { return p.reverse ? L - 1 - t : t; };
        load_act<T, R>(p.x, b, d, pos(t0), dir, true, 0, L - t0, run);
#pragma unroll
        for (int i = 0; i < R; ++i) x[3 + i] = run[i];
#pragma unroll
        for (int m = 0; m < 6; ++m) {
            const int i = m < 3 ? m : R + m, t = t0 - 3 + i;
            float one[1] = {0.f};
            if (t >= 0) load_act<T, 1>(p.x, b, d, pos(t), dir, true, 0, t < L ? 1 : 0, one);
            else one[0] = conv_hist<T>(p, b, d, t);
            x[i] = one[0];
        }
        const int64_t o = (int64_t)b * p.sdo.b + (int64_t)d * p.sdo.c + (int64_t)pos(t0) * p.sdo.p;
        const int64_t os = dir * p.sdo.p;
        if (p.dout32) load_run<float, R>(static_cast<const float*>(p.dout) + o, os, 0, L - t0, run);
        else load_run<T, R>(static_cast<const T*>(p.dout) + o, os, 0, L - t0, run);
#pragma unroll
        for (int i = 0; i < R + 3; ++i) {
            if (i < R) dp[i] = run[i < R ? i : 0];
            else if (t0 + i >= L) dp[i] = 0.f;
            else dp[i] = p.dout32 ? static_cast<const float*>(p.dout)[o + i * os]
                                  : Elem<T>::to_f(static_cast<const T*>(p.dout)[o + i * os]);
        }
        float dx[R + 3];                                       // dx[t0 - 3 .. t0 + 7]
#pragma unroll
        for (int i = 0; i < R + 3; ++i) dx[i] = 0.f;
#pragma unroll
        for (int i = 0; i < R + 3; ++i) {
            const int sn = p.since && t0 + i < L ? p.since[t0 + i] : 4;
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
                    if (i - lag < R) dx[3 + i - lag < R + 3 ? 3 + i - lag : 0] += w[lag] * dp[i];
                    if (i < R) sw[lag] = fmaf(dp[i], x[3 + i - lag], sw[lag]);
                }
            if (i < R) sw[4] += dp[i];
        }
#pragma unroll
        for (int i = 0; i < R; ++i) run[i] = dx[3 + i];
        store_run<T, R>(static_cast<T*>(p.dx) + (int64_t)b * p.sdx.b + (int64_t)d * p.sdx.c +
                            (int64_t)pos(t0) * p.sdx.p,
                        dir * p.sdx.p, 0, L - t0, run);
        if (t0 == 0 && p.dhist)
#pragma unroll
            for (int m = 0; m < 3; ++m)                        // positions -3 .. -1
                if (m >= 4 - p.width)
                    static_cast<T*>(p.dhist)[rowid * (p.width - 1) + (p.width - 4 + m)] =
                        Elem<T>::from_f(dx[m]);
    }
    __shared__ float red[kConvRowThreads / 32][5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o /= 2) sw[k] += __shfl_xor_sync(0xffffffffu, sw[k], o);
        if (threadIdx.x % 32 == 0) red[threadIdx.x / 32][k] = sw[k];
    }
    __syncthreads();
    if (threadIdx.x < 5) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kConvRowThreads / 32; ++i) v += red[i][threadIdx.x];
        p.part[(((int64_t)b * p.chunks + blockIdx.x) * p.dim + d) * 5 + threadIdx.x] = v;
    }
}

template <typename T>
__global__ void __launch_bounds__(128) conv_bwd_cl_kernel(const ConvBwdParams p) {
    constexpr int E = kConvClRun;
    const int L = p.seqlen, dir = p.reverse ? -1 : 1;
    const int d = (blockIdx.x * blockDim.x + threadIdx.x) * E;
    const int b = blockIdx.y, chunk = blockIdx.z;
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
    auto load_x = [&](int t, float (&v)[E]) {
        if (t >= 0) {
            load_act<T, E>(p.x, b, d, pos(t), dir, false, 0, t < L ? hi : 0, v);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = i < hi ? conv_hist<T>(p, b, d + i, t) : 0.f;
        }
    };
    // xw[lag] holds x_{t-lag}; before the first step x_{tb-1-lag}
#pragma unroll
    for (int lag = 0; lag < 3; ++lag) load_x(tb - 1 - lag, xw[lag]);
#pragma unroll 4
    for (int t = tb; t < te + 3; ++t) {
        float x[E], dp[E];
        load_x(t, x);
        const int64_t o = (int64_t)b * p.sdo.b + (int64_t)d * p.sdo.c + (int64_t)pos(t) * p.sdo.p;
        const int h = t < L ? hi : 0;
        if (p.dout32) load_run<float, E>(static_cast<const float*>(p.dout) + o, p.sdo.c, 0, h, dp);
        else load_run<T, E>(static_cast<const T*>(p.dout) + o, p.sdo.c, 0, h, dp);
        const int sn = p.since && t < L ? p.since[t] : 4;
        float out[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            xw[3][i] = xw[2][i];
            xw[2][i] = xw[1][i];
            xw[1][i] = xw[0][i];
            xw[0][i] = x[i];
            acc[3][i] = acc[2][i];                             // acc[lag]: dx_{t-lag} so far
            acc[2][i] = acc[1][i];
            acc[1][i] = acc[0][i];
            acc[0][i] = 0.f;
            if (p.silu) {
                float pre = bias[i];
#pragma unroll
                for (int lag = 0; lag < 4; ++lag)
                    if (lag <= sn) pre = fmaf(w[lag][i], xw[lag][i], pre);
                dp[i] *= dsilu(pre);
            }
#pragma unroll
            for (int lag = 0; lag < 4; ++lag)
                if (lag <= sn) {
                    acc[lag][i] = fmaf(w[lag][i], dp[i], acc[lag][i]);
                    if (t < te) sw[lag][i] = fmaf(dp[i], xw[lag][i], sw[lag][i]);
                }
            if (t < te) sw[4][i] += dp[i];
            out[i] = acc[3][i];
        }
        const int s = t - 3;                                   // dx_s is complete
        if (s >= tb) {
            store_run<T, E>(static_cast<T*>(p.dx) + (int64_t)b * p.sdx.b + (int64_t)d * p.sdx.c +
                                (int64_t)pos(s) * p.sdx.p,
                            p.sdx.c, 0, hi, out);
        } else if (chunk == 0 && p.dhist && s >= -(p.width - 1)) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (i < hi)
                    static_cast<T*>(p.dhist)[((int64_t)b * p.dim + d + i) * (p.width - 1) +
                                             (p.width - 1 + s)] = Elem<T>::from_f(out[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < hi)
#pragma unroll
            for (int k = 0; k < 5; ++k)
                p.part[(((int64_t)b * p.chunks + chunk) * p.dim + d + i) * 5 + k] = sw[k][i];
}

// dw (dim, width), dbias (dim) from the partial rows (rows, dim, 5: by lag, then bias).
__global__ void __launch_bounds__(128) conv_reduce_kernel(const ConvReduceParams p) {
    const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= (int64_t)p.dim * 5) return;
    const int d = (int)(idx / 5), k = (int)(idx % 5);
    float v = 0.f;
#pragma unroll 8
    for (int64_t r = 0; r < p.rows; ++r) v += p.part[r * p.dim * 5 + idx];
    if (k < 4) {
        if (p.dw && k < p.width) p.dw[(int64_t)d * p.width + p.width - 1 - k] = v;
    } else if (p.dbias) {
        p.dbias[d] = v;
    }
}

}  // namespace ssm
