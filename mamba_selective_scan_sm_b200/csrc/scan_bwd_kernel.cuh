// The gradient of the selective scan for sm_100a.
//
// With a_t = exp(delta_t A) (0 at a packed sequence's first step), per (batch row, channel
// d, state n) and in scan order t:
//   h_t   = a_t h_{t-1} + delta_t u_t B_t              (recomputed)
//   lam_t = g_t C_t + a_{t+1} lam_{t+1},  g = dy silu(z), lam past the end = d final state
//   dC_t  = sum_d g_t h_t             dB_t = sum_d lam_t delta_t u_t
//   dA    = sum_t q_t delta_t         q_t = lam_t a_t h_{t-1}
//   du    = D g + delta sum_n lam B   ddelta = u sum_n lam B + sum_n q A
//   dz    = dy (C.h + D u) silu'(z)   d h_0 = a_0 lam_0
// and d dt = ddelta sigmoid(dt + bias) under the softplus.
//
// The recurrence cannot be run backwards from its last state (dividing by a small a_t loses
// everything), so a forward pass first leaves the state before every 8th step in global
// memory (MODE kCheckpoint: 8 bytes per channel and step at d_state 16), and the backward
// sweep redoes 8 steps at a time from there with a_t and h_t in registers. Two exps per
// (channel, step, state) in all. A grid too small for the GPU splits the sequence into
// segments: a first pass (MODE kSummary) reduces each to its decay product, its end state
// from zero and its adjoint carry from zero, and scan_bwd_carry_kernel chains them.
//
// Roles. A lane holds 4 states (two fp32 pairs) of a channel, S = d_state / 4 lanes a
// channel, 32 / S channels a warp (KC times, one after the other). A CTA of 4 warps stages a
// tile of TT steps for its G channels in shared memory (delta, delta u, g per channel and
// step; B and C as fp32 rows), its warps run the recurrences, and the CTA then writes the
// tile's gradients. Sums over states (y, sum lam B, sum q A) and over a warp's channels (dB,
// dC) are transpose-reductions by shuffles: each level halves the values a lane carries.
// dB and dC are summed over the CTA's channels in shared memory and over the CTAs by
// scan_bwd_reduce_bc_kernel from one partial row per CTA: no atomics, so the sums come out
// in the same order every time.
#pragma once

#include "bwd_params.h"
#include "device_common.cuh"

namespace ssm {

constexpr int kBwdWarps = 4;
constexpr int kBwdThreads = 32 * kBwdWarps;
constexpr int kCheckpoint = 0, kSummary = 1;
constexpr float kLn2 = 0.6931471805599453f;

// Static shape of the kernels for S lanes per channel.
template <int S> struct BwdShape {
    static constexpr int NS = 4 * S;                           // states, padded
    static constexpr int CW = 32 / S;                          // channels per warp and slot
    static constexpr int KC = S <= 4 ? 1 : S / 4;              // channel slots per warp
    static constexpr int G = kBwdWarps * CW * KC;              // channels per CTA
    static constexpr int TT = S == 4 ? 32 : (S == 2 || S == 8) ? 16 : 8;   // steps per tile
    static constexpr int NSUB = TT / kSubSteps;
    static constexpr int EPT = G * TT / kBwdThreads;           // elements per thread and tensor
    static constexpr int RB = NS + 4;                          // row of B / C in floats
    // shared memory, in floats
    static constexpr int kSt = 4 * G * (TT + 1);               // {delta, delta u, g, start}
    static constexpr int kU = G * (TT + 1);
    static constexpr int kOut = G * (TT + 2);                  // one of y, s1, s2
    static constexpr int kBC = TT * RB;
    static constexpr int kPart = kBwdWarps * TT * 2 * NS;
    static constexpr int kPrm = 8 * G;
    static constexpr int kSum = 2 * G * TT;                    // channel-last dD, dbias sums
    static constexpr int kCarry = KC > 2 ? kBwdThreads * KC * 8 : 0;
};

// f[i] = element lo..hi-1 of a run (others 0) at p + i * step; one 16-byte (or two, or one
// 8-byte) load when the run is dense, whole and aligned, in either direction.
template <typename T, int N>
__device__ __forceinline__ void load_run(const T* p, int64_t step, int lo, int hi, float (&f)[N]) {
    constexpr int BY = N * (int)sizeof(T);
    if constexpr (BY >= 8) {
        constexpr int V = BY >= 16 ? 16 : 8;
        const T* q = step < 0 ? p - (N - 1) : p;
        if (lo <= 0 && hi >= N && (step == 1 || step == -1) &&
            (reinterpret_cast<uintptr_t>(q) & (V - 1)) == 0) {
            alignas(16) T e[N];
            if constexpr (V == 16) {
#pragma unroll
                for (int k = 0; k < BY / 16; ++k)
                    reinterpret_cast<uint4*>(e)[k] = reinterpret_cast<const uint4*>(q)[k];
            } else {
                *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(q);
            }
            if (step > 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = Elem<T>::to_f(e[i]);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = Elem<T>::to_f(e[N - 1 - i]);
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = i >= lo && i < hi ? Elem<T>::to_f(p[(int64_t)i * step]) : 0.f;
}

template <typename T, int N>
__device__ __forceinline__ void store_run(T* p, int64_t step, int lo, int hi, const float (&f)[N]) {
    constexpr int BY = N * (int)sizeof(T);
    if constexpr (BY >= 8) {
        constexpr int V = BY >= 16 ? 16 : 8;
        T* q = step < 0 ? p - (N - 1) : p;
        if (lo <= 0 && hi >= N && (step == 1 || step == -1) &&
            (reinterpret_cast<uintptr_t>(q) & (V - 1)) == 0) {
            alignas(16) T e[N];
            if (step > 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) e[i] = Elem<T>::from_f(f[i]);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) e[N - 1 - i] = Elem<T>::from_f(f[i]);
            }
            if constexpr (V == 16) {
#pragma unroll
                for (int k = 0; k < BY / 16; ++k)
                    reinterpret_cast<uint4*>(q)[k] = reinterpret_cast<uint4*>(e)[k];
            } else {
                *reinterpret_cast<uint2*>(q) = *reinterpret_cast<uint2*>(e);
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i >= lo && i < hi) p[(int64_t)i * step] = Elem<T>::from_f(f[i]);
}

// A run of N elements of an activation, along positions (alongp: from channel c, position
// pos, positions going by dir) or along channels (from channel c at position pos). Elements
// lo..hi-1 exist; the others read 0.
template <typename T, int N>
__device__ __forceinline__ void load_act(const ActIn& a, int b, int c, int pos, int dir,
                                         bool alongp, int lo, int hi, float (&f)[N]) {
    const int64_t off = (int64_t)b * a.s.b + (int64_t)c * a.s.c + (int64_t)pos * a.s.p;
    const int64_t step = alongp ? dir * a.s.p : a.s.c;
    if (!a.scale) {
        load_run<T, N>(static_cast<const T*>(a.p) + off, step, lo, hi, f);
        return;
    }
    const int8_t* q = static_cast<const int8_t*>(a.p) + off;
    const float* sc = a.scale + (int64_t)b * a.ss.b;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        f[i] = 0.f;
        if (i >= lo && i < hi) {
            const int pi = alongp ? pos + dir * i : pos, ci = alongp ? c : c + i;
            f[i] = (float)q[(int64_t)i * step] *
                   sc[(int64_t)ci * a.ss.c + (int64_t)(pi / kBlock8) * a.ss.p];
        }
    }
}

__device__ __forceinline__ float sigmoidf_(float v) {
    return __fdividef(1.f, 1.f + ex2(-v * kLog2e));
}

// Sum over the S lanes of a channel of 8 values a lane (one per step): every level adds
// the partner's half of the values still carried. Afterwards a lane holds 8 / min(S, 8)
// sums, those of the steps from reduce8_first(lane).
template <int S>
__device__ __forceinline__ void reduce8(float (&v)[8], int lane) {
    int cnt = 8;
#pragma unroll
    for (int w = 1; w < S; w *= 2) {
        if (cnt > 1) {
            cnt /= 2;
            const bool up = lane & w;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < cnt) {
                    const float send = up ? v[k] : v[k + cnt];
                    const float keep = up ? v[k + cnt] : v[k];
                    v[k] = keep + __shfl_xor_sync(0xffffffffu, send, w);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
        }
    }
}
template <int S>
__device__ __forceinline__ int reduce8_first(int lane) {
    int off = 0, cnt = 8;
#pragma unroll
    for (int w = 1; w < S && w < 8; w *= 2) {
        cnt /= 2;
        off += (lane & w) ? cnt : 0;
    }
    return off;
}

// Sum over the 32 / S channels of a warp of 32 values a lane (8 steps x 4 states):
// afterwards a lane holds S sums, values reduce32_first(lane) and on.
template <int S>
__device__ __forceinline__ void reduce32(float (&v)[32], int lane) {
    int cnt = 32;
#pragma unroll
    for (int w = S; w < 32; w *= 2) {
        cnt /= 2;
        const bool up = lane & w;
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (k < cnt) {
                const float send = up ? v[k] : v[k + cnt];
                const float keep = up ? v[k + cnt] : v[k];
                v[k] = keep + __shfl_xor_sync(0xffffffffu, send, w);
            }
    }
}
template <int S>
__device__ __forceinline__ int reduce32_first(int lane) {
    int off = 0, cnt = 32;
#pragma unroll
    for (int w = S; w < 32; w *= 2) {
        cnt /= 2;
        off += (lane & w) ? cnt : 0;
    }
    return off;
}

// Where a thread's run of EPT elements of a tile lies: along the steps of one channel, or
// (channel-last) along the channels of one step.
template <int S, bool CL> struct BwdRun {
    using H = BwdShape<S>;
    int ch, tl;
    __device__ BwdRun(int tid) {
        if (CL) {
            tl = tid / (H::G / H::EPT);
            ch = tid % (H::G / H::EPT) * H::EPT;
        } else {
            ch = tid / (H::TT / H::EPT);
            tl = tid % (H::TT / H::EPT) * H::EPT;
        }
    }
    __device__ __forceinline__ int c(int i) const { return CL ? ch + i : ch; }
    __device__ __forceinline__ int t(int i) const { return CL ? tl : tl + i; }
};

// Per-channel constants in shared memory: 4 right-aligned taps, conv bias, dt bias, D.
template <int S>
__device__ __forceinline__ void load_prm(const BwdParams& p, int d0, float* prm) {
    using H = BwdShape<S>;
    for (int c = threadIdx.x; c < H::G; c += kBwdThreads) {
        const int d = d0 + c;
        const bool in = d < p.dim;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int kk = k - (4 - p.conv_width);
            prm[c * 8 + k] = in && p.conv_w && kk >= 0 ? p.conv_w[(int64_t)d * p.conv_width + kk] : 0.f;
        }
        prm[c * 8 + 4] = in && p.conv_w && p.conv_b ? p.conv_b[d] : 0.f;
        prm[c * 8 + 5] = in && p.dbias ? p.dbias[d] : 0.f;
        prm[c * 8 + 6] = in && p.D ? p.D[d] : 0.f;
    }
}

// Stage steps [t0, t0 + TT) (scan order) of the CTA's channels: {delta, delta u, g, start}
// per channel and step, u where ADJ, and the rows of B (and C where ADJ). Steps past the
// end and channels past dim stage zeros: a = 1 and no input, which leave both recurrences
// where they are.
template <typename T, int S, bool CL, bool ADJ>
__device__ __forceinline__ void stage_tile(const BwdParams& p, int b, int d0, int t0,
                                           const float* prm, float4* st, float* us, float* Bs,
                                           float* Cs) {
    using H = BwdShape<S>;
    constexpr int E = H::EPT;
    const int tid = threadIdx.x, L = p.seqlen, dir = p.reverse ? -1 : 1;
    const BwdRun<S, CL> r(tid);
    const int d = d0 + r.ch, t = t0 + r.tl;
    const int pos = p.reverse ? L - 1 - t : t;
    // valid elements of the run: [0, hi)
    const int hi = CL ? (t < L ? min(E, p.dim - d) : 0) : (d < p.dim ? min(E, L - t) : 0);
    float u[E], dt[E], g[E];
    if (p.conv_w) {
        float acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = prm[r.c(i) * 8 + 4];
        if constexpr (CL) {
            const int sn = p.since && t < L ? p.since[t] : 4;
            for (int lag = 0; lag < p.conv_width; ++lag) {
                if (lag > sn) break;
                float x[E];
                if (t - lag >= 0) {
                    load_act<T, E>(p.x, b, d, pos - dir * lag, dir, false, 0, hi, x);
                } else {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const T* h = static_cast<const T*>(p.hist);
                        x[i] = h && i < hi ? Elem<T>::to_f(h[((int64_t)b * p.dim + d + i) * (p.conv_width - 1) +
                                                            (p.conv_width - 1 + t - lag)])
                                           : 0.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < E; ++i) acc[i] = fmaf(prm[r.c(i) * 8 + 3 - lag], x[i], acc[i]);
            }
        } else {
            float x[E], xh[3];                                 // the run, and the 3 steps before
            load_act<T, E>(p.x, b, d, pos, dir, true, 0, hi, x);
#pragma unroll
            for (int m = 0; m < 3; ++m) {
                const int tm = t - 3 + m;
                xh[m] = 0.f;
                if (hi > 0 && 3 - m < p.conv_width) {
                    if (tm >= 0) {
                        float one[1];
                        load_act<T, 1>(p.x, b, d, pos - dir * (3 - m), dir, true, 0, 1, one);
                        xh[m] = one[0];
                    } else if (p.hist && tm >= -(p.conv_width - 1)) {
                        xh[m] = Elem<T>::to_f(static_cast<const T*>(
                            p.hist)[((int64_t)b * p.dim + d) * (p.conv_width - 1) + (p.conv_width - 1 + tm)]);
                    }
                }
            }
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = prm[r.ch * 8 + k];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int sn = p.since && i < hi ? p.since[t + i] : 4;
#pragma unroll
                for (int lag = 0; lag < 4; ++lag) {
                    const float v = i >= lag ? x[i >= lag ? i - lag : 0] : xh[i >= lag ? 0 : 3 + i - lag];
                    if (lag <= sn) acc[i] = fmaf(w[3 - lag], v, acc[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < E; ++i) u[i] = i < hi ? silu(acc[i]) : 0.f;
    } else {
        load_act<T, E>(p.x, b, d, pos, dir, !CL, 0, hi, u);
    }
    load_act<T, E>(p.dt, b, d, pos, dir, !CL, 0, hi, dt);
    if constexpr (ADJ) {
        const T* dy = static_cast<const T*>(p.dy) + (int64_t)b * p.sdy.b + (int64_t)d * p.sdy.c +
                      (int64_t)pos * p.sdy.p;
        load_run<T, E>(dy, CL ? p.sdy.c : dir * p.sdy.p, 0, hi, g);
        if (p.z.p) {
            float z[E];
            load_act<T, E>(p.z, b, d, pos, dir, !CL, 0, hi, z);
#pragma unroll
            for (int i = 0; i < E; ++i) g[i] *= silu(z[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float raw = dt[i] + prm[r.c(i) * 8 + 5];
        float dl = p.softplus ? (raw > 20.f ? raw : softplus(raw)) : raw;
        if (i >= hi) dl = 0.f;
        const float start = p.since && i < hi && p.since[t0 + r.t(i)] == 0 ? -INFINITY : 0.f;
        st[r.c(i) * (H::TT + 1) + r.t(i)] = make_float4(dl, dl * u[i], ADJ ? g[i] : 0.f, start);
        if constexpr (ADJ) us[r.c(i) * (H::TT + 1) + r.t(i)] = u[i];
    }
    // rows of B and C
    const T* Bp = static_cast<const T*>(p.Bm) + (int64_t)b * p.sB.b;
    const T* Cp = static_cast<const T*>(p.Cm) + (int64_t)b * p.sC.b;
#pragma unroll 4
    for (int k = tid; k < H::NS * H::TT; k += kBwdThreads) {
        const int n = CL ? k % H::NS : k / H::TT, tl = CL ? k / H::NS : k % H::TT;
        const int tt = t0 + tl, ps = p.reverse ? L - 1 - tt : tt;
        const bool in = n < p.dstate && tt < L;
        Bs[tl * H::RB + n] = in ? Elem<T>::to_f(Bp[(int64_t)n * p.sB.c + (int64_t)ps * p.sB.p]) : 0.f;
        if constexpr (ADJ)
            Cs[tl * H::RB + n] = in ? Elem<T>::to_f(Cp[(int64_t)n * p.sC.c + (int64_t)ps * p.sC.p]) : 0.f;
    }
}

// A of one lane's 4 states (times log2 e), zeros past dim or d_state.
template <int S, bool HEADS>
__device__ __forceinline__ void load_A(const BwdParams& p, int d, int j, uint64_t (&A2)[2]) {
    float a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int n = 4 * j + k;
        const bool in = d < p.dim && n < p.dstate;
        a[k] = !in ? 0.f : kLog2e * (HEADS ? p.A[d / p.head_dim] : p.A[(int64_t)d * p.dstate + n]);
    }
    A2[0] = pk2(a[0], a[1]);
    A2[1] = pk2(a[2], a[3]);
}

// Decay of one step for a lane's 4 states: 2^(delta A log2 e + start), start = -inf at a
// sequence's first step. With A per head one exp serves all.
template <bool HEADS>
__device__ __forceinline__ void decay(const uint64_t (&A2)[2], float dl, float start, uint64_t (&a)[2]) {
    if constexpr (HEADS) {
        const float e = ex2(fmaf(dl, lo2(A2[0]), start));
        a[0] = a[1] = pk2(e, e);
    } else {
        const uint64_t d2 = pk2(dl, dl), o2 = pk2(start, start);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 x = upk2(fma2(d2, A2[k], o2));
            a[k] = pk2(ex2(x.x), ex2(x.y));
        }
    }
}

__device__ __forceinline__ void ldpair(const float* s, uint64_t (&v)[2]) {
    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(s);
    v[0] = q.x;
    v[1] = q.y;
}
__device__ __forceinline__ void stpair(float* s, const uint64_t (&v)[2]) {
    *reinterpret_cast<ulonglong2*>(s) = make_ulonglong2(v[0], v[1]);
}

// Four states of a (batch, dim, dstate) tensor, zeros past dim or d_state or when null.
__device__ __forceinline__ void load_state(const BwdParams& p, const float* s, int b, int d, int j,
                                           uint64_t (&v)[2]) {
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int n = 4 * j + k;
        f[k] = s && d < p.dim && n < p.dstate ? s[((int64_t)b * p.dim + d) * p.dstate + n] : 0.f;
    }
    v[0] = pk2(f[0], f[1]);
    v[1] = pk2(f[2], f[3]);
}

// Offset of a lane's 4 states in a (rows, dim, NS) scratch array.
template <int S>
__device__ __forceinline__ int64_t ns_off(const BwdParams& p, int64_t row, int d, int j) {
    return (row * p.dim + d) * (4 * S) + 4 * j;
}

// The forward pass: checkpoints of the state (MODE kCheckpoint), or a segment's summary.
template <typename T, int S, bool CL, bool HEADS, int MODE>
__global__ void __launch_bounds__(kBwdThreads) scan_bwd_states_kernel(const BwdParams p) {
    using H = BwdShape<S>;
    constexpr bool SUM = MODE == kSummary;
    extern __shared__ __align__(16) float sm[];
    float4* st = reinterpret_cast<float4*>(sm);
    float* us = sm + H::kSt;
    float* Bs = us + (SUM ? H::kU : 0);
    float* Cs = Bs + H::kBC;
    float* prm = Cs + (SUM ? H::kBC : 0);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int j = lane % S, cl = lane / S;
    const int b = blockIdx.y, d0 = blockIdx.x * H::G, seg = blockIdx.z;
    const int tb = seg * p.seg_len, te = min(p.seqlen, tb + p.seg_len);
    const int64_t row = (int64_t)seg * p.batch + b;
    load_prm<S>(p, d0, prm);
    uint64_t h[H::KC][2], A2[H::KC][2], R[H::KC][2], P[H::KC][2];
#pragma unroll
    for (int kc = 0; kc < H::KC; ++kc) {
        const int d = d0 + (warp * H::KC + kc) * H::CW + cl;
        load_A<S, HEADS>(p, d, j, A2[kc]);
        R[kc][0] = R[kc][1] = 0;
        P[kc][0] = P[kc][1] = pk2(1.f, 1.f);
        h[kc][0] = h[kc][1] = 0;
        if (!SUM && seg == 0) load_state(p, p.h0, b, d, j, h[kc]);
        if (!SUM && seg > 0 && d < p.dim) ldpair(p.sumS + ns_off<S>(p, row, d, j), h[kc]);
    }
    for (int t0 = tb; t0 < te; t0 += H::TT) {
        __syncthreads();
        stage_tile<T, S, CL, SUM>(p, b, d0, t0, prm, st, us, Bs, Cs);
        __syncthreads();
#pragma unroll
        for (int kc = 0; kc < H::KC; ++kc) {
            const int c = (warp * H::KC + kc) * H::CW + cl, d = d0 + c;
            const float4* srow = st + c * (H::TT + 1);
#pragma unroll 1
            for (int sub = 0; sub < H::NSUB; ++sub) {
                if (!SUM && d < p.dim)
                    stpair(p.ckpt + ns_off<S>(p, (int64_t)b * p.nsub + t0 / kSubSteps + sub, d, j), h[kc]);
#pragma unroll
                for (int i = 0; i < kSubSteps; ++i) {
                    const int tl = sub * kSubSteps + i;
                    const float4 s = srow[tl];
                    uint64_t a[2], bv[2], cv[2];
                    decay<HEADS>(A2[kc], s.x, s.w, a);
                    ldpair(Bs + tl * H::RB + 4 * j, bv);
                    if (SUM) ldpair(Cs + tl * H::RB + 4 * j, cv);
                    const uint64_t du2 = pk2(s.y, s.y), g2 = pk2(s.z, s.z);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        h[kc][k] = fma2(a[k], h[kc][k], mul2(du2, bv[k]));
                        if (SUM) {
                            P[kc][k] = mul2(P[kc][k], a[k]);
                            R[kc][k] = fma2(P[kc][k], mul2(g2, cv[k]), R[kc][k]);
                        }
                    }
                }
            }
        }
    }
    if (SUM) {
#pragma unroll
        for (int kc = 0; kc < H::KC; ++kc) {
            const int d = d0 + (warp * H::KC + kc) * H::CW + cl;
            if (d < p.dim) {
                const int64_t o = ns_off<S>(p, row, d, j);
                stpair(p.sumP + o, P[kc]);
                stpair(p.sumS + o, h[kc]);
                stpair(p.sumR + o, R[kc]);
            }
        }
    }
}

// Chains the segments' summaries: sumS[seg] becomes the state before the segment, sumR[seg]
// the adjoint carry a_t lam_t from behind it. One thread per (batch row, channel, state).
template <int NS>
__global__ void __launch_bounds__(256) scan_bwd_carry_kernel(const BwdParams p) {
    const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t per = (int64_t)p.batch * p.dim * NS;
    if (idx >= per) return;
    const int n = (int)(idx % NS);
    const int64_t bd = idx / NS;
    float h = p.h0 && n < p.dstate ? p.h0[bd * p.dstate + n] : 0.f;
    float m = p.dhl && n < p.dstate ? p.dhl[bd * p.dstate + n] : 0.f;
    for (int s = 0; s < p.nseg; ++s) {
        const int64_t o = s * per + idx;
        const float pr = p.sumP[o], e = p.sumS[o];
        p.sumS[o] = h;
        h = fmaf(pr, h, e);
    }
    for (int s = p.nseg - 1; s >= 0; --s) {
        const int64_t o = s * per + idx;
        const float pr = p.sumP[o], r = p.sumR[o];
        p.sumR[o] = m;
        m = fmaf(pr, m, r);
    }
}

// The backward sweep.
template <typename T, int S, bool CL, bool HEADS>
__global__ void __launch_bounds__(kBwdThreads) scan_bwd_kernel(const BwdParams p) {
    using H = BwdShape<S>;
    constexpr int KC = H::KC, TT = H::TT, E = H::EPT;
    constexpr bool REGS = KC <= 2;                             // m and dA of every slot in registers
    extern __shared__ __align__(16) float sm[];
    float4* st = reinterpret_cast<float4*>(sm);
    float* us = sm + H::kSt;
    float* ys = us + H::kU;
    float* s1s = ys + H::kOut;
    float* s2s = s1s + H::kOut;
    float* Bs = s2s + H::kOut;
    float* Cs = Bs + H::kBC;
    float* part = Cs + H::kBC;
    float* prm = part + H::kPart;
    float* carry = prm + H::kPrm;
    float* sums = carry + H::kCarry;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int j = lane % S, cl = lane / S;
    const int b = blockIdx.y, d0 = blockIdx.x * H::G, seg = blockIdx.z;
    const int L = p.seqlen, tb = seg * p.seg_len, te = min(L, tb + p.seg_len);
    const int64_t row = (int64_t)seg * p.batch + b;
    load_prm<S>(p, d0, prm);

    uint64_t m[REGS ? KC : 1][2], dA[REGS ? KC : 1][2], A2[REGS ? KC : 1][2];
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) {
        const int d = d0 + (warp * KC + kc) * H::CW + cl;
        const int r = REGS ? kc : 0;
        dA[r][0] = dA[r][1] = 0;
        m[r][0] = m[r][1] = 0;
        if (te == L) load_state(p, p.dhl, b, d, j, m[r]);
        else if (d < p.dim) ldpair(p.sumR + ns_off<S>(p, row, d, j), m[r]);
        if constexpr (REGS) {
            load_A<S, HEADS>(p, d, j, A2[r]);
        } else {
            stpair(carry + ((size_t)kc * kBwdThreads + tid) * 8, m[0]);
            stpair(carry + ((size_t)kc * kBwdThreads + tid) * 8 + 4, dA[0]);
        }
    }
    const BwdRun<S, CL> run(tid);
    float dD = 0.f, dBias = 0.f;
    if constexpr (CL) {
        for (int k = tid; k < H::kSum; k += kBwdThreads) sums[k] = 0.f;
    }

    const int ntiles = (te - tb + TT - 1) / TT;
    for (int tile = ntiles - 1; tile >= 0; --tile) {
        const int t0 = tb + tile * TT;
        __syncthreads();
        stage_tile<T, S, CL, true>(p, b, d0, t0, prm, st, us, Bs, Cs);
        __syncthreads();
#pragma unroll 1
        for (int sub = H::NSUB - 1; sub >= 0; --sub) {
            float vB[32], vC[32];
            if constexpr (KC > 1) {
#pragma unroll
                for (int i = 0; i < 32; ++i) vB[i] = vC[i] = 0.f;
            }
            constexpr int UNR = REGS ? KC : 1;
#pragma unroll UNR
            for (int kc = 0; kc < KC; ++kc) {
                const int c = (warp * KC + kc) * H::CW + cl, d = d0 + c;
                const int r = REGS ? kc : 0;
                uint64_t h0[2] = {0, 0};
                if (d < p.dim)
                    ldpair(p.ckpt + ns_off<S>(p, (int64_t)b * p.nsub + t0 / kSubSteps + sub, d, j), h0);
                if constexpr (!REGS) {
                    load_A<S, HEADS>(p, d, j, A2[0]);
                    ldpair(carry + ((size_t)kc * kBwdThreads + tid) * 8, m[0]);
                    ldpair(carry + ((size_t)kc * kBwdThreads + tid) * 8 + 4, dA[0]);
                }
                const float4* srow = st + c * (TT + 1) + sub * kSubSteps;
                const float* Br = Bs + sub * kSubSteps * H::RB + 4 * j;
                const float* Cr = Cs + sub * kSubSteps * H::RB + 4 * j;
                uint64_t a[kSubSteps][2], h[kSubSteps][2];
#pragma unroll
                for (int i = 0; i < kSubSteps; ++i) {
                    const float4 s = srow[i];
                    uint64_t bv[2];
                    decay<HEADS>(A2[r], s.x, s.w, a[i]);
                    ldpair(Br + i * H::RB, bv);
                    const uint64_t du2 = pk2(s.y, s.y);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        h[i][k] = fma2(a[i][k], i ? h[i ? i - 1 : 0][k] : h0[k], mul2(du2, bv[k]));
                }
                float y[8], s1[8], s2[8];
#pragma unroll
                for (int i = kSubSteps - 1; i >= 0; --i) {
                    const float4 s = srow[i];
                    uint64_t bv[2], cv[2], lam[2], q[2];
                    ldpair(Br + i * H::RB, bv);
                    ldpair(Cr + i * H::RB, cv);
                    const uint64_t d2 = pk2(s.x, s.x), du2 = pk2(s.y, s.y), g2 = pk2(s.z, s.z);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        lam[k] = fma2(g2, cv[k], m[r][k]);
                        m[r][k] = mul2(a[i][k], lam[k]);
                        q[k] = mul2(m[r][k], i ? h[i ? i - 1 : 0][k] : h0[k]);
                        dA[r][k] = fma2(q[k], d2, dA[r][k]);
                        const int v = 4 * i + 2 * k;
                        float2 fb, fc;                         // summed over the warp's slots
                        if constexpr (KC > 1) {
                            fb = upk2(fma2(lam[k], du2, pk2(vB[v], vB[v + 1])));
                            fc = upk2(fma2(g2, h[i][k], pk2(vC[v], vC[v + 1])));
                        } else {
                            fb = upk2(mul2(lam[k], du2));
                            fc = upk2(mul2(g2, h[i][k]));
                        }
                        vB[v] = fb.x;
                        vB[v + 1] = fb.y;
                        vC[v] = fc.x;
                        vC[v + 1] = fc.y;
                    }
                    const float2 fy = upk2(fma2(cv[1], h[i][1], mul2(cv[0], h[i][0])));
                    const float2 f1 = upk2(fma2(bv[1], lam[1], mul2(bv[0], lam[0])));
                    y[i] = fy.x + fy.y;
                    s1[i] = f1.x + f1.y;
                    if constexpr (HEADS) {
                        const float2 f2 = upk2(add2(q[0], q[1]));
                        s2[i] = lo2(A2[r][0]) * (f2.x + f2.y);
                    } else {
                        const float2 f2 = upk2(fma2(q[1], A2[r][1], mul2(q[0], A2[r][0])));
                        s2[i] = f2.x + f2.y;
                    }
                }
                reduce8<S>(y, lane);
                reduce8<S>(s1, lane);
                reduce8<S>(s2, lane);
                if (j < 8) {
                    const int o = c * (TT + 2) + sub * kSubSteps + reduce8_first<S>(lane);
                    constexpr int CNT = S >= 8 ? 1 : 8 / S;
#pragma unroll
                    for (int k = 0; k < CNT; ++k) {
                        ys[o + k] = y[k];
                        s1s[o + k] = s1[k];
                        s2s[o + k] = s2[k];
                    }
                }
                if constexpr (!REGS) {
                    stpair(carry + ((size_t)kc * kBwdThreads + tid) * 8, m[0]);
                    stpair(carry + ((size_t)kc * kBwdThreads + tid) * 8 + 4, dA[0]);
                }
            }
            reduce32<S>(vB, lane);
            reduce32<S>(vC, lane);
            const int first = reduce32_first<S>(lane);
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const int v = first + k, tl = sub * kSubSteps + v / 4, n = 4 * j + v % 4;
                float* o = part + ((warp * TT + tl) * 2) * H::NS + n;
                o[0] = vB[k];
                o[H::NS] = vC[k];
            }
        }
        __syncthreads();
        // the tile's gradients, one run per thread
        {
            const int d = d0 + run.ch, t = t0 + run.tl, dir = p.reverse ? -1 : 1;
            const int pos = p.reverse ? L - 1 - t : t;
            const int hi = CL ? (t < L ? min(E, p.dim - d) : 0) : (d < p.dim ? min(E, L - t) : 0);
            if (hi > 0) {
                float dt[E], z[E], dy[E], du[E], ddt[E], dz[E];
                load_act<T, E>(p.dt, b, d, pos, dir, !CL, 0, hi, dt);
                if (p.z.p) {
                    load_act<T, E>(p.z, b, d, pos, dir, !CL, 0, hi, z);
                    load_run<T, E>(static_cast<const T*>(p.dy) + (int64_t)b * p.sdy.b +
                                       (int64_t)d * p.sdy.c + (int64_t)pos * p.sdy.p,
                                   CL ? p.sdy.c : dir * p.sdy.p, 0, hi, dy);
                }
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int c = run.c(i), tl = run.t(i), o = c * (TT + 2) + tl;
                    const float4 s = st[c * (TT + 1) + tl];
                    const float u = us[c * (TT + 1) + tl], Dv = prm[c * 8 + 6];
                    const float s1 = s1s[o], s2 = s2s[o] * kLn2;
                    du[i] = fmaf(s.z, Dv, s.x * s1);
                    const float ddelta = fmaf(u, s1, s2);
                    ddt[i] = p.softplus ? ddelta * sigmoidf_(dt[i] + prm[c * 8 + 5]) : ddelta;
                    if (p.z.p) {
                        const float sg = sigmoidf_(z[i]);
                        dz[i] = dy[i] * fmaf(Dv, u, ys[o]) * (sg * fmaf(z[i], 1.f - sg, 1.f));
                    }
                    if (CL) {
                        if (i < hi) {
                            sums[c * TT + tl] += s.z * u;
                            sums[H::G * TT + c * TT + tl] += ddt[i];
                        }
                    } else if (i < hi) {
                        dD = fmaf(s.z, u, dD);
                        dBias += ddt[i];
                    }
                }
                auto at = [&](const Str& s) {
                    return (int64_t)b * s.b + (int64_t)d * s.c + (int64_t)pos * s.p;
                };
                auto step = [&](const Str& s) { return CL ? s.c : dir * s.p; };
                if (p.du32) store_run<float, E>(p.du32 + at(p.sdu), step(p.sdu), 0, hi, du);
                else store_run<T, E>(static_cast<T*>(p.du) + at(p.sdu), step(p.sdu), 0, hi, du);
                store_run<T, E>(static_cast<T*>(p.ddt) + at(p.sddt), step(p.sddt), 0, hi, ddt);
                if (p.z.p && p.dz)
                    store_run<T, E>(static_cast<T*>(p.dz) + at(p.sdz), step(p.sdz), 0, hi, dz);
            }
        }
        // the CTA's dB and dC of the tile
        {
            constexpr int ROW = 2 * H::NS;
            float* out = p.parts + (((int64_t)blockIdx.x * p.batch + b) * L + t0) * ROW;
            const int n = min(TT, te - t0) * ROW;
            for (int k = tid; k < n; k += kBwdThreads) {
                float v = part[k];
#pragma unroll
                for (int w = 1; w < kBwdWarps; ++w) v += part[w * TT * ROW + k];
                out[k] = v;
            }
        }
    }
    // what the sweep summed over its steps
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) {
        const int d = d0 + (warp * KC + kc) * H::CW + cl;
        const int r = REGS ? kc : 0;
        if constexpr (!REGS) {
            ldpair(carry + ((size_t)kc * kBwdThreads + tid) * 8, m[0]);
            ldpair(carry + ((size_t)kc * kBwdThreads + tid) * 8 + 4, dA[0]);
        }
        if (d < p.dim) {
            stpair(p.pA + ns_off<S>(p, row, d, j), dA[r]);
            if (seg == 0 && p.dh0) {
                const float2 lo = upk2(m[r][0]), hi = upk2(m[r][1]);
                const float f[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (4 * j + k < p.dstate) p.dh0[((int64_t)b * p.dim + d) * p.dstate + 4 * j + k] = f[k];
            }
        }
    }
    __syncthreads();
    if constexpr (!CL) {
        // the threads of a channel are neighbours within a warp (TT / EPT of them)
        constexpr int PER = TT / E;
#pragma unroll
        for (int w = 1; w < PER; w *= 2) {
            dD += __shfl_xor_sync(0xffffffffu, dD, w);
            dBias += __shfl_xor_sync(0xffffffffu, dBias, w);
        }
        if (tid % PER == 0 && d0 + run.ch < p.dim) {
            float* o = p.pD + (row * p.dim + d0 + run.ch) * 2;
            o[0] = dD;
            o[1] = dBias;
        }
    } else {
        for (int c = tid; c < H::G; c += kBwdThreads) {
            if (d0 + c >= p.dim) break;
            float v0 = 0.f, v1 = 0.f;
            for (int t = 0; t < TT; ++t) {
                v0 += sums[c * TT + t];
                v1 += sums[H::G * TT + c * TT + t];
            }
            float* o = p.pD + (row * p.dim + d0 + c) * 2;
            o[0] = v0;
            o[1] = v1;
        }
    }
}

}  // namespace ssm
