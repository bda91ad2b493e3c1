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
// everything), so a forward pass first leaves the state before every T-th step (4, or 8 up to
// d_state 8) in global memory (MODE kCheckpoint), and the backward sweep redoes T steps at a
// time from there with a_t and h_t in registers. Two exps per (channel, step, state) in all. A
// grid too small for the GPU splits the sequence into segments: a first pass (MODE kSummary)
// reduces each to its decay product, its end state from zero and its adjoint carry from zero,
// and scan_bwd_carry_kernel chains them.
//
// Roles. A lane holds 4 states (two fp32 pairs) of KL channels, S = d_state / 4 lanes a
// channel: B and C are read once for both channels, and their dB and dC add up before a
// shuffle. W scan warps run the recurrences of one staged tile of TT steps (delta, delta u, g
// per channel and step; B and C as fp32 rows) while NH helper threads finish the tile before
// it (the gradients' elementwise part, stores) and stage the one after it, whose inputs
// asynchronous copies brought a tile earlier. One CTA barrier a tile.
// Sums over states (y, sum lam B, sum q A) and over a warp's channels (dB, dC) are
// transpose-reductions by shuffles; the lanes hold their states and channels in orders that
// make most rounds exchange the same register everywhere (slot_order, BwdShape::channel). dB
// and dC are summed over the CTA's warps in shared memory and over the CTAs by
// scan_bwd_reduce_bc_kernel from one partial row per CTA: no atomics, so the sums come out in
// the same order every time.
//
// What bounds it (B8 D1536 L2048 N16 bf16 + conv: 0.26 ms checkpoints, 0.65 ms sweep): latency.
// 384 CTAs give an SM five scan warps, which issue 0.25 instructions a cycle each through
// dependent exps, multiplies and shuffles; issue slots 48 % busy, shared memory 60 %, DRAM
// 17 %. Measured otherwise, sweep alone: every warp both staging and scanning one channel per
// lane 0.79 ms, two channels per lane 0.92 (fewer instructions, half the warps); tiles of 8
// steps 0.69; two sub-tiles in hand per scan warp 1.10 (spills).
#pragma once

#include <type_traits>

#include "bwd_params.h"
#include "device_common.cuh"

namespace ssm {

constexpr int kCheckpoint = 0, kSummary = 1;
constexpr float kLn2 = 0.6931471805599453f;

// A sum of many terms: the fp32 sum and, beside it, the sum of what its additions rounded off
// (exact, by the two-sum). A plain fp32 sum of terms of one sign loses 2^-25 of itself per
// addition: over 2^19 steps 0.5 %.
struct LongSum {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float t = hi + x, b = t - hi;
        lo += (hi - (t - b)) + (x - b);
        hi = t;
    }
    __device__ __forceinline__ float get() const {             // (an infinity stays one)
        return fabsf(lo) < INFINITY ? hi + lo : hi;
    }
};
constexpr int kDrainSteps = 512;  // steps between two additions to the long sums

// Static shape of the kernels for S lanes per channel.
template <int S> struct BwdShape {
    static constexpr int NS = 4 * S;                           // states, padded
    static constexpr int CW = 32 / S;                          // channels per warp and slot
    static constexpr int KL = S >= 4 ? 2 : 1;                  // channels a lane takes in step
    static constexpr int T = 8 / KL;                           // steps in registers
    static constexpr int W = S == 4 ? 2 : 4;                   // scan warps per CTA
    static constexpr int NH = S == 1 || S == 2 ? 128 : 64;     // helper threads
    static constexpr int NT = 32 * W + NH;
    static constexpr int CTAS = S == 4 ? 3 : S >= 8 ? 2 : 1;   // per SM, by registers (see BwdSmem)
    static constexpr int KC = S <= 8 ? 1 : S / 8;              // such groups a warp takes in turn
    static constexpr int NC = CW < 4 ? CW : 4;                 // state orders (see slot_order)
    static constexpr int G = W * CW * KL * KC;                 // channels per CTA
    static constexpr int TT = S == 4 ? 16 : 8;                 // steps per tile
    static constexpr int NSUB = TT / T;
    static constexpr int DRAIN = kDrainSteps / TT;             // tiles
    static constexpr int EPT = G * TT / NH;                    // elements per helper and tensor
    static constexpr int RB = NS;                              // row of B / C in floats
    // shared memory, in floats
    // one of two staged tiles
    static constexpr int kSt = 2 * G * (TT + 1);               // {delta, delta u}
    static constexpr int kG = G * (TT + 1);
    static constexpr int RO = TT + 1;                          // row of u, y, s1, s2 in floats
    static constexpr int kU = G * RO;
    static constexpr int kOut = G * RO;                        // one of y, s1, s2
    static constexpr int RQ = TT * RB + 16;                    // one order's copy of B / C: the copies
    static constexpr int kBC = NC * RQ;                        // begin 16 banks apart
    static constexpr int kDecay = G * (TT + 1);                // A per head: decays
    static constexpr int kStaged(bool adj, bool heads) {
        return kSt + (heads ? kDecay : 0) + (adj ? kG + kU + 2 * kBC : kBC);
    }
    static constexpr int RP = 2 * NS + 8;                      // row of dB, dC of a step
    static constexpr int PS = S >= 16 || S == 4 ? T : TT; // steps of dB, dC summed at a time
    static constexpr int kPart = W * PS * RP;
    static constexpr int kPrm = 8 * G;
    static constexpr int kMask = 4;                            // sequence starts of the two tiles, as bits
    static constexpr int kSum = 2 * G * TT;                    // channel-last dD, dbias sums
    static constexpr int kCarry = KC > 1 ? 32 * W * KC * KL * 8 : 0;
    // the place in the CTA of channel kl of lane (warp, cl, j) in group kc. Lanes with odd j
    // take their two channels the other way round: the sums over a channel's lanes then
    // exchange the same slot in every lane (reduce_states).
    static __device__ __forceinline__ int channel(int warp, int kc, int cl, int j, int kl) {
        return ((warp * KC + kc) * CW + cl) * KL + (KL > 1 && S > 1 ? kl ^ (j & 1) : kl);
    }
};

// The order of a lane's 4 states. Slot k of a channel's lane j holds state 4 j + (k ^ q),
// q = the low bits of the channel's place in its warp. Two lanes whose channels differ in
// bit 1 of q then hold each other's second pair of states in their first pair of slots, and
// two that differ in bit 0 each other's odd state in the even slot: the sums over a warp's
// channels exchange the same slots in every lane, without a select per value (measured with
// the selects: 33 instructions per channel, step and state; without: see scan_bwd_kernel).
// Everything the kernels pass to one another in scratch memory is in this order. A lane's two
// channels (KL) have the same order.
template <int S>
__device__ __forceinline__ int slot_order(int d) {
    return d / BwdShape<S>::KL & (BwdShape<S>::NC - 1);        // CTAs begin at multiples of G
}

// One tile's inputs as they lie in global memory, copied to shared memory a tile ahead of
// their use (two buffers): rows of positions (x with a halo for the conv in front, or behind
// in the reverse direction), or channel-last rows of channels in scan order (x with 3 steps
// before it).
template <typename T, int S, bool CL> struct BwdRaw {
    using H = BwdShape<S>;
    static constexpr int ES = (int)sizeof(T);
    static constexpr int kXRow = CL ? H::G * ES : 16 + H::TT * ES;
    static constexpr int kRow = CL ? H::G * ES : H::TT * ES;
    static constexpr int kBRow = CL ? (H::NS * ES < 16 ? 16 : H::NS * ES) : H::TT * ES;
    static constexpr int kRows = CL ? H::TT : H::G;
    static constexpr int X = 0;
    static constexpr int DT = X + (CL ? H::TT + 3 : H::G) * kXRow;
    static constexpr int Z = DT + kRows * kRow;
    static constexpr int DY = Z + kRows * kRow;
    static constexpr int B = DY + kRows * kRow;
    static constexpr int C = B + (CL ? H::TT : H::NS) * kBRow;
    static constexpr int SINCE = C + (CL ? H::TT : H::NS) * kBRow;
    static constexpr int SC = SINCE + 16;                      // 8 bits: scales, 3 tensors x 2 blocks x G
    static constexpr int bytes(bool q8) { return SC + (q8 ? 6 * H::G * 4 : 0); }
};

// The first hi of N dense elements from p on (others 0): 16-byte loads when all of them are there
// and aligned.
template <typename T, int N>
__device__ __forceinline__ void load_run(const T* p, int hi, float (&f)[N]) {
    constexpr int BY = N * (int)sizeof(T);
    static_assert(BY % 16 == 0, "runs of whole 16-byte units");
    if (hi >= N && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        alignas(16) T e[N];
#pragma unroll
        for (int k = 0; k < BY / 16; ++k) reinterpret_cast<uint4*>(e)[k] = reinterpret_cast<const uint4*>(p)[k];
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = Elem<T>::to_f(e[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = i < hi ? Elem<T>::to_f(p[i]) : 0.f;
}

template <typename T, int N>
__device__ __forceinline__ void store_run(T* p, int hi, const float (&f)[N]) {
    constexpr int BY = N * (int)sizeof(T);
    static_assert(BY % 16 == 0, "runs of whole 16-byte units");
    if (hi >= N && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        alignas(16) T e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = Elem<T>::from_f(f[i]);
#pragma unroll
        for (int k = 0; k < BY / 16; ++k) reinterpret_cast<uint4*>(p)[k] = reinterpret_cast<uint4*>(e)[k];
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < hi) p[i] = Elem<T>::from_f(f[i]);
}

// One element of an activation: channel c, position pos of batch row b.
template <typename T>
__device__ __forceinline__ float load_act(const ActIn& a, int b, int c, int pos) {
    const int64_t off = (int64_t)b * a.s.b + (int64_t)c * a.s.c + (int64_t)pos * a.s.p;
    if (!a.scale) return Elem<T>::to_f(static_cast<const T*>(a.p)[off]);
    return (float)static_cast<const int8_t*>(a.p)[off] *
           a.scale[(int64_t)b * a.ss.b + (int64_t)c * a.ss.c + (int64_t)(pos / kBlock8) * a.ss.p];
}

// 1 / (1 + e^-v) by the SFU's exp and its division (2 ulp each) and the exponent's rounding, which
// is |v| 2^-24 of e^-v: relative 3e-7 for v > -1, 1e-6 at -16. The gates' and the softplus'
// derivatives take it, once per element and not in the recurrence, beside the forward's silu of
// the same making; a full-precision exp and division would be 20 instructions more an element.
__device__ __forceinline__ float sigmoidf_(float v) {
    return __fdividef(1.f, 1.f + ex2(-v * kLog2e));
}

// Sums over the S lanes of a channel of 8 values a lane, [channel][step]. With two channels
// the first level trades the second slot (lanes with odd j hold the channels the other way
// round); every further level adds the partner's half of the steps still carried.
// Afterwards a lane holds kept() sums of its first slot's channel, from step first() on.
template <int S> struct StateSums {
    using H = BwdShape<S>;
    static constexpr bool kTrade = H::KL == 2 && S > 1;
    static constexpr int levels() {
        int n = 0;
        for (int w = kTrade ? 2 : 1; w < S; w *= 2) ++n;
        return n;
    }
    static constexpr int kept() { return levels() >= (H::T == 8 ? 3 : 2) ? 1 : H::T >> levels(); }
    static __device__ __forceinline__ void sum(float (&v)[8], int lane) {
        if constexpr (kTrade) {
#pragma unroll
            for (int i = 0; i < H::T; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[H::T + i], 1);
        }
        int cnt = H::T;
#pragma unroll
        for (int w = kTrade ? 2 : 1; w < S; w *= 2) {
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
    static __device__ __forceinline__ int first(int lane) {
        int off = 0, cnt = H::T;
#pragma unroll
        for (int w = kTrade ? 2 : 1; w < S; w *= 2)
            if (cnt > 1) {
                cnt /= 2;
                off += (lane & w) ? cnt : 0;
            }
        return off;
    }
};

// Sum over the first NC channels of a lane's 4 values (one per state slot): each level
// adds the partner's other half. Leaves 4 / NC values, of slots 0, 4 / NC, ...
template <int S>
__device__ __forceinline__ void reduce_slots(const uint64_t (&v)[2], float* r) {
    constexpr int NC = BwdShape<S>::NC;
    const float2 a = upk2(v[0]), b = upk2(v[1]);
    if constexpr (NC == 4) {
        const float2 c = upk2(add2(v[0], pk2(__shfl_xor_sync(0xffffffffu, b.x, 2 * S),
                                             __shfl_xor_sync(0xffffffffu, b.y, 2 * S))));
        r[0] = c.x + __shfl_xor_sync(0xffffffffu, c.y, S);
    } else if constexpr (NC == 2) {
        r[0] = a.x + __shfl_xor_sync(0xffffffffu, a.y, S);
        r[1] = b.x + __shfl_xor_sync(0xffffffffu, b.y, S);
    } else {
        r[0] = a.x;
        r[1] = a.y;
        r[2] = b.x;
        r[3] = b.y;
    }
}

// Sum over the remaining 32 / S / 4 groups of channels of T values (one per step), over the
// upper lane bits: a lane keeps kept() of them from step first() on.
template <int S> struct GroupSums {
    static constexpr int T = BwdShape<S>::T;
    static constexpr int kept() {
        int n = T;
        for (int w = 4 * S; w < 32; w *= 2) n /= 2;
        return n;
    }
    static __device__ __forceinline__ void sum(float (&v)[T], int lane) {
        int cnt = T;
#pragma unroll
        for (int w = 4 * S; w < 32; w *= 2) {
            cnt /= 2;
            const bool up = lane & w;
#pragma unroll
            for (int k = 0; k < T / 2; ++k)
                if (k < cnt) {
                    const float send = up ? v[k] : v[k + cnt];
                    const float keep = up ? v[k + cnt] : v[k];
                    v[k] = keep + __shfl_xor_sync(0xffffffffu, send, w);
                }
        }
    }
    static __device__ __forceinline__ int first(int lane) {
        int off = 0, cnt = T;
#pragma unroll
        for (int w = 4 * S; w < 32; w *= 2) {
            cnt /= 2;
            off += (lane & w) ? cnt : 0;
        }
        return off;
    }
};

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

// Per-channel constants in shared memory: 4 right-aligned taps, conv bias, dt bias, D, and A
// where it is per head.
template <int S>
__device__ __forceinline__ void load_prm(const BwdParams& p, int d0, float* prm) {
    using H = BwdShape<S>;
    for (int c = threadIdx.x; c < H::G; c += H::NT) {
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
        prm[c * 8 + 7] = in && p.head_dim ? p.A[d / p.head_dim] : 0.f;
    }
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int have) {
    // BYTES (4, 8 or 16) to shared memory, the first `have` of them from src, zeros behind
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
                 "r"(have));
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// One asynchronous copy of a tile, worked out once: its source advances with the tile.
struct __align__(16) BwdCopy {
    const uint8_t* src;           // the row (position 0), or channel-last the unit of the row
    uint32_t step;                // channel-last: bytes between positions / 16; else log2 of the element size
    uint16_t dst;                 // in the buffer
    int8_t at;                    // position relative to the tile's lowest, or step to its first
    int8_t bytes;                 // that exist (zeros are filled in behind); < 0: no copy
};

template <typename T, int S, bool CL, bool Q8, bool ADJ> struct BwdCopies {
    using H = BwdShape<S>;
    using R = BwdRaw<T, S, CL>;
    static constexpr int TT = H::TT, ES = R::ES, EQ = Q8 ? 1 : ES;     // EQ: of x, delta, z
    // bytes of a copy and copies of a row, for rows of x, delta, z (Q), dout and B, C
    static constexpr int UQ = !CL && TT * EQ < 16 ? TT * EQ : 16;
    static constexpr int PQ = CL ? H::G * EQ / 16 : TT * EQ / UQ;
    static constexpr int PY = CL ? H::G * ES / 16 : TT * ES / 16;
    static constexpr int PB = CL ? (H::NS * ES + 15) / 16 : TT * ES / 16;
    static constexpr int NX = CL ? (TT + 3) * PQ : H::G * PQ;
    static constexpr int NQ = CL ? TT * PQ : H::G * PQ;
    static constexpr int NH = CL ? 0 : H::G;                           // halos of x
    static constexpr int NB = CL ? TT * PB : H::NS * PB;
    static constexpr int NY = CL ? TT * PY : H::G * PY;
    // x, halo, delta, B (and with ADJ z, dout, C)
    static constexpr int COUNT = NX + NH + NQ + NB + (ADJ ? NQ + NY + NB : 0);
    static constexpr int PER = (COUNT + H::NH - 1) / H::NH;

    static __device__ BwdCopy make(const BwdParams& p, int b, int d0, int id) {
        const int have = p.dim - d0;
        auto rows = [&](const void* q, const Str& st, int first, int count, int e, int unit, int per, int i,
                        int off, int drow) {
            // positions of row i / per
            const int r = i / per, k = i % per;
            const uint8_t* src = static_cast<const uint8_t*>(q) + ((int64_t)b * st.b + (int64_t)(first + (r < count ? r : 0)) * st.c) * e;
            return BwdCopy{src, (uint32_t)(e == 4 ? 2 : e - 1), (uint16_t)(off + r * drow + k * unit),
                           (int8_t)(k * (unit / e)), (int8_t)(r < count ? unit : 0)};
        };
        auto steps = [&](const void* q, const Str& st, int first, int count, int e, int per, int i, int lead,
                         int off, int drow) {
            const int r = i / per, k = i % per;
            const uint8_t* src = static_cast<const uint8_t*>(q) + ((int64_t)b * st.b + first) * e + k * 16;
            const int n = min(16, max(0, count * e - 16 * k));
            return BwdCopy{src, (uint32_t)(st.p * e / 16), (uint16_t)(off + r * drow + k * 16),
                           (int8_t)(r - lead), (int8_t)n};
        };
        auto act = [&](const ActIn& a, int i, int off) {
            if constexpr (CL) return steps(a.p, a.s, d0, have, EQ, PQ, i, 0, off, R::kRow);
            else return rows(a.p, a.s, d0, have, EQ, UQ, PQ, i, off, R::kRow);
        };
        auto bc = [&](const void* q, const Str& st, int i, int off) {
            if constexpr (CL) return steps(q, st, 0, p.dstate, ES, PB, i, 0, off, R::kBRow);
            else return rows(q, st, 0, p.dstate, ES, 16, PB, i, off, R::kBRow);
        };
        const BwdCopy none{nullptr, 0, 0, 0, -1};
        if (id < NX) {
            if constexpr (CL) {
                return id / PQ < 3 && !p.conv_w ? none : steps(p.x.p, p.x.s, d0, have, EQ, PQ, id, 3, R::X, R::kXRow);
            } else {
                return rows(p.x.p, p.x.s, d0, have, EQ, UQ, PQ, id, R::X + (p.reverse ? 0 : 16), R::kXRow);
            }
        }
        id -= NX;
        if (id < NH) {
            if (!p.conv_w) return none;
            BwdCopy c = rows(p.x.p, p.x.s, d0, have, EQ, UQ, 1, id, R::X + (p.reverse ? TT * EQ : 16 - UQ), R::kXRow);
            c.at = (int8_t)(p.reverse ? TT : -(UQ / EQ));
            return c;
        }
        id -= NH;
        if (id < NQ) return act(p.dt, id, R::DT);
        id -= NQ;
        if (id < NB) return bc(p.Bm, p.sB, id, R::B);
        id -= NB;
        if (!ADJ) return none;
        if (id < NQ) return p.z.p ? act(p.z, id, R::Z) : none;
        id -= NQ;
        if (id < NY) {
            if constexpr (CL) return steps(p.dy, p.sdy, d0, have, ES, PY, id, 0, R::DY, R::kRow);
            else return rows(p.dy, p.sdy, d0, have, ES, 16, PY, id, R::DY, R::kRow);
        }
        id -= NY;
        return id < NB ? bc(p.Cm, p.sC, id, R::C) : none;
    }
};

// Shared memory of the sweep, and the CTAs that an SM holds with it: of fp32 d_state 9 to 16 (91 to
// 101 KB) and of A per head there (77 to 81 KB in bf16) two instead of three, of fp32 d_state 65
// to 128 (135 to 139 KB) one instead of two.
template <typename T, int S, bool CL, bool Q8, bool HEADS> struct BwdSmem {
    using H = BwdShape<S>;
    static constexpr int kHead = (H::kPrm + H::kMask) * 4;
    static constexpr int kRaw = BwdRaw<T, S, CL>::bytes(Q8);
    static constexpr int kSweep =
        (2 * H::kStaged(true, HEADS) + 6 * H::kOut + H::kPart + H::kCarry + (CL ? H::kSum : 0)) * 4 + kHead +
        3 * kRaw + BwdCopies<T, S, CL, Q8, true>::COUNT * 16;
    static constexpr int kPerSM = 228 * 1024, kReserved = 1024;   // an SM's, and of it the system's per CTA
    static constexpr int kFit = kPerSM / (kSweep + kReserved);
    static constexpr int CTAS = H::CTAS < kFit ? H::CTAS : kFit;
    static_assert(CTAS >= 1, "a CTA fits an SM");
};

// The plain form of the same copies, element by element, for rows that are not aligned.
template <typename T, int S, bool CL, bool Q8, bool ADJ>
__device__ __forceinline__ void fetch_plain(const BwdParams& p, int hid, int b, int d0, int t0, uint8_t* raw) {
    using H = BwdShape<S>;
    using R = BwdRaw<T, S, CL>;
    constexpr int TT = H::TT, ES = R::ES, EQ = Q8 ? 1 : ES;
    const int L = p.seqlen, pos0 = p.reverse ? L - t0 - TT : t0, have = p.dim - d0;
    auto put = [&](uint8_t* dst, int k, const uint8_t* q, bool in, auto size) {
        constexpr int e = decltype(size)::value;
        if constexpr (e == 4) reinterpret_cast<uint32_t*>(dst)[k] = in ? *reinterpret_cast<const uint32_t*>(q) : 0u;
        else if constexpr (e == 2) reinterpret_cast<uint16_t*>(dst)[k] = in ? *reinterpret_cast<const uint16_t*>(q) : 0;
        else dst[k] = in ? *q : 0;
    };
    // `rows` rows of `width` elements; which of a row and its column is the position goes by CL
    auto copy = [&](const void* ptr, const Str& st, int first, int count, int rows, int width, int lead,
                    uint8_t* dst, int drow, auto size) {
        constexpr int e = decltype(size)::value;
        const uint8_t* src = static_cast<const uint8_t*>(ptr) + (int64_t)b * st.b * e;
#pragma unroll 2
        for (int i = hid; i < rows * width; i += H::NH) {
            const int r = i / width, k = i % width, t = t0 - lead + r;
            const int pos = CL ? (p.reverse ? L - 1 - t : t) : pos0 + k, c = CL ? k : r;
            const bool in = c < count && pos >= 0 && pos < L;
            put(dst + r * drow, k, src + ((int64_t)(first + c) * st.c + (int64_t)pos * st.p) * e, in, size);
        }
    };
    std::integral_constant<int, EQ> sq;
    std::integral_constant<int, ES> se;
    constexpr int ROWS = CL ? TT : H::G, WIDTH = CL ? H::G : TT;
    if constexpr (CL) {
        copy(p.x.p, p.x.s, d0, have, TT + 3, H::G, 3, raw + R::X, R::kXRow, sq);
    } else {
        copy(p.x.p, p.x.s, d0, have, H::G, TT, 0, raw + R::X + (p.reverse ? 0 : 16), R::kXRow, sq);
        const uint8_t* src = static_cast<const uint8_t*>(p.x.p) + ((int64_t)b * p.x.s.b + (int64_t)d0 * p.x.s.c) * EQ;
        for (int i = hid; i < (p.conv_w ? H::G * 4 : 0); i += H::NH) {
            const int r = i / 4, o = i % 4 - 4, t = t0 + o, pos = p.reverse ? L - 1 - t : t;
            put(raw + R::X + r * R::kXRow, p.reverse ? TT - 1 - o : 16 / EQ + o,
                src + ((int64_t)r * p.x.s.c + pos) * EQ, r < have && pos >= 0 && pos < L, sq);
        }
    }
    copy(p.dt.p, p.dt.s, d0, have, ROWS, WIDTH, 0, raw + R::DT, R::kRow, sq);
    copy(p.Bm, p.sB, 0, p.dstate, CL ? TT : H::NS, CL ? H::NS : TT, 0, raw + R::B, R::kBRow, se);
    if constexpr (ADJ) {
        if (p.z.p) copy(p.z.p, p.z.s, d0, have, ROWS, WIDTH, 0, raw + R::Z, R::kRow, sq);
        copy(p.dy, p.sdy, d0, have, ROWS, WIDTH, 0, raw + R::DY, R::kRow, se);
        copy(p.Cm, p.sC, 0, p.dstate, CL ? TT : H::NS, CL ? H::NS : TT, 0, raw + R::C, R::kBRow, se);
    }
}

// Start copying the inputs of steps [t0, t0 + TT) into a buffer: x, delta, B, and with ADJ z,
// dout, C. Asynchronous copies where the host found every row aligned to their units
// (p.async), from the CTA's table; else plain loads.
template <typename T, int S, bool CL, bool Q8, bool ADJ>
__device__ __forceinline__ void fetch_tile(const BwdParams& p, const BwdCopy* table, int hid, int b, int d0, int t0,
                                           uint8_t* raw) {
    using H = BwdShape<S>;
    using R = BwdRaw<T, S, CL>;
    using K = BwdCopies<T, S, CL, Q8, ADJ>;
    const int L = p.seqlen, pos0 = p.reverse ? L - t0 - H::TT : t0;
    if (p.async) {
        const uint32_t dst = smem_u32(raw);
#pragma unroll
        for (int k = 0; k < K::PER; ++k) {
            const int id = hid + k * H::NH;
            if (id >= K::COUNT) break;
            const BwdCopy c = table[id];
            const int pos = CL ? (p.reverse ? L - 1 - (t0 + c.at) : t0 + c.at) : pos0 + c.at;
            const int n = pos >= 0 && pos < L ? c.bytes : 0;
            const uint8_t* src = c.src + (n <= 0 ? 0 : CL ? (int64_t)pos * c.step * 16 : (int64_t)pos << c.step);
            if (c.bytes < 0) continue;
            // units of 8 bytes are those of 8-bit rows in 8-step tiles
            if (K::UQ == 8 && id < K::NX + K::NH + K::NQ) cp_async<8>(dst + c.dst, src, n);
            else if (K::UQ == 8 && ADJ && id >= K::NX + K::NH + K::NQ + K::NB && id < K::NX + K::NH + 2 * K::NQ + K::NB)
                cp_async<8>(dst + c.dst, src, n);
            else cp_async<16>(dst + c.dst, src, n);
        }
    } else {
        fetch_plain<T, S, CL, Q8, ADJ>(p, hid, b, d0, t0, raw);
    }
    if constexpr (Q8) {
        // a tile and its halo span at most two blocks of 64 positions: both their scales
        const int have = p.dim - d0, last = (L - 1) / kBlock8;
        const int lo = min(max(pos0 - 3, 0) / kBlock8, last), hi = min(max(pos0 + H::TT + 2, 0) / kBlock8, last);
        for (int i = hid; i < 6 * H::G; i += H::NH) {
            const int c = i % H::G, which = i / H::G, k = which / 2;
            const ActIn& a = k == 0 ? p.x : k == 1 ? p.dt : p.z;
            const bool in = c < have && a.scale && (k < 2 || ADJ);
            const float* q = in ? a.scale + (int64_t)b * a.ss.b + (int64_t)(d0 + c) * a.ss.c +
                                      (int64_t)(which % 2 ? hi : lo) * a.ss.p
                                : p.x.scale;
            cp_async<4>(smem_u32(raw + R::SC + 4 * i), q, in ? 4 : 0);
        }
    }
    if (p.since && hid == 0) cp_async<H::TT>(smem_u32(raw + R::SINCE), p.since + t0, H::TT);
    cp_async_commit();
}

// N elements at p (dense, aligned to their size together), reversed if rev.
template <typename T, int N>
__device__ __forceinline__ void take_run(const T* p, bool rev, float (&f)[N]) {
    constexpr int BY = N * (int)sizeof(T);
    constexpr int V = BY >= 16 ? 16 : BY;
    alignas(16) T e[N];
#pragma unroll
    for (int k = 0; k < BY / V; ++k) {
        if constexpr (V == 16) reinterpret_cast<uint4*>(e)[k] = reinterpret_cast<const uint4*>(p)[k];
        else if constexpr (V == 8) reinterpret_cast<uint2*>(e)[k] = reinterpret_cast<const uint2*>(p)[k];
        else if constexpr (V == 4) reinterpret_cast<uint32_t*>(e)[k] = reinterpret_cast<const uint32_t*>(p)[k];
        else reinterpret_cast<uint16_t*>(e)[k] = reinterpret_cast<const uint16_t*>(p)[k];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const T v = rev ? e[N - 1 - i] : e[i];
        if constexpr (sizeof(T) == 1) f[i] = (float)v;
        else f[i] = Elem<T>::to_f(v);
    }
}

// The first hi values of a run, to p (dense): from p on, or (rev) from p + N - 1 backwards.
// vec: such runs are aligned to their size.
template <typename T, int N>
__device__ __forceinline__ void put_run(T* p, bool rev, bool vec, int hi, const float (&f)[N]) {
    constexpr int BY = N * (int)sizeof(T), V = BY >= 16 ? 16 : 8;
    static_assert(BY % V == 0, "whole units");
    if (vec && hi == N) {
        alignas(16) T e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = Elem<T>::from_f(rev ? f[N - 1 - i] : f[i]);
#pragma unroll
        for (int k = 0; k < BY / V; ++k) {
            if constexpr (V == 16) reinterpret_cast<uint4*>(p)[k] = reinterpret_cast<uint4*>(e)[k];
            else reinterpret_cast<uint2*>(p)[k] = reinterpret_cast<uint2*>(e)[k];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < hi) p[rev ? N - 1 - i : i] = Elem<T>::from_f(f[i]);
}

// A thread's run of EPT values of x, delta or z (which = 0, 1, 2; codes where packed) or of
// dout (which = 3), in scan order; for x shift steps earlier (channel-last only).
template <typename T, int S, bool CL, bool Q8>
__device__ __forceinline__ void take(const BwdParams& p, const uint8_t* raw, int which,
                                     const BwdRun<S, CL>& r, int t0, float (&f)[BwdShape<S>::EPT],
                                     int shift = 0) {
    using H = BwdShape<S>;
    using R = BwdRaw<T, S, CL>;
    constexpr int E = H::EPT;
    const bool q8 = Q8 && which < 3, rev = !CL && p.reverse;
    const uint8_t* row = raw + (which == 0 ? R::X + (CL ? (r.tl + 3 - shift) * R::kXRow : r.ch * R::kXRow + (p.reverse ? 0 : 16))
                                : (which == 1 ? R::DT : which == 2 ? R::Z : R::DY) + (CL ? r.tl : r.ch) * R::kRow);
    const int at = CL ? r.ch : rev ? H::TT - E - r.tl : r.tl;
    if (!q8) {
        take_run<T, E>(reinterpret_cast<const T*>(row) + at, rev, f);
        return;
    }
    take_run<int8_t, E>(reinterpret_cast<const int8_t*>(row) + at, rev, f);
    const float* sc = reinterpret_cast<const float*>(raw + R::SC) + which * 2 * H::G;
    const int pos0 = p.reverse ? p.seqlen - t0 - H::TT : t0;
    const int lo = max(pos0 - 3, 0) / kBlock8;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int t = t0 + r.t(i) - shift, pos = p.reverse ? p.seqlen - 1 - t : t;
        f[i] *= sc[(pos / kBlock8 == lo ? 0 : H::G) + r.c(i)];
    }
}

// out[i] = f(in[i]), two at a time.
template <int E, typename F>
__device__ __forceinline__ void each_pair(float (&out)[E], const float (&in)[E], F&& f) {
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        const float2 v = upk2(f(pk2(in[i], in[i + 1])));
        out[i] = v.x;
        out[i + 1] = v.y;
    }
}

// Turn a tile's raw inputs into what the recurrences take: delta and delta u per channel and
// step, g and u where ADJ, and the rows of B (and C
// where ADJ) in each order of the states. Steps past the end and channels past dim get
// zeros: a = 1 and no input, which leave both recurrences where they are.
template <typename T, int S, bool CL, bool Q8, bool ADJ, bool HEADS>
__device__ __forceinline__ void stage_tile(const BwdParams& p, int hid, int b, int d0, int t0, const uint8_t* raw,
                                           const float* prm, float2* st, float* as, float* gs,
                                           float* us, float* Bs, float* Cs, uint32_t* mask) {
    using H = BwdShape<S>;
    using R = BwdRaw<T, S, CL>;
    constexpr int E = H::EPT;
    const int tid = hid, L = p.seqlen;
    const BwdRun<S, CL> r(tid);
    const int d = d0 + r.ch, t = t0 + r.tl;
    // valid elements of the run: [0, hi)
    const int hi = CL ? (t < L ? min(E, p.dim - d) : 0) : (d < p.dim ? min(E, L - t) : 0);
    const uint8_t* since = raw + R::SINCE;
    float u[E], dt[E], g[E];
    take<T, S, CL, Q8>(p, raw, 0, r, t0, u);
    if (p.conv_w) {
        float acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = prm[r.c(i) * 8 + 4];
        // x at scan position tm < 0 of channel c: the history
        auto past = [&](int c, int tm) {
            return p.hist && d0 + c < p.dim && tm >= -(p.conv_width - 1)
                       ? Elem<T>::to_f(static_cast<const T*>(
                             p.hist)[((int64_t)b * p.dim + d0 + c) * (p.conv_width - 1) + (p.conv_width - 1 + tm)])
                       : 0.f;
        };
        if constexpr (CL) {
            const int sn = min(p.since ? since[r.tl] : 4, p.conv_width - 1);   // the furthest tap
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = fmaf(prm[r.c(i) * 8 + 3], u[i], acc[i]);
#pragma unroll
            for (int lag = 1; lag < 4; ++lag) {
                float x[E];
                take<T, S, CL, Q8>(p, raw, 0, r, t0, x, lag);
                if (t - lag < 0)
#pragma unroll
                    for (int i = 0; i < E; ++i) x[i] = past(r.ch + i, t - lag);
                if (lag <= sn)
#pragma unroll
                    for (int i = 0; i < E; ++i) acc[i] = fmaf(prm[r.c(i) * 8 + 3 - lag], x[i], acc[i]);
            }
        } else {
            float xh[3], h0[2], h1[2];                         // the 3 steps before the run
            const uint8_t* row = raw + R::X + r.ch * R::kXRow;
            using Q = std::conditional_t<Q8, int8_t, T>;
            const Q* e = reinterpret_cast<const Q*>(row) + (p.reverse ? H::TT - r.tl : 16 / (int)sizeof(Q) + r.tl - 4);
            take_run<Q, 2>(e, false, h0);
            take_run<Q, 2>(e + 2, false, h1);
            xh[0] = p.reverse ? h1[0] : h0[1];
            xh[1] = p.reverse ? h0[1] : h1[0];
            xh[2] = p.reverse ? h0[0] : h1[1];
            if constexpr (Q8) {
                const float* sc = reinterpret_cast<const float*>(raw + R::SC);
                const int pos0 = p.reverse ? L - t0 - H::TT : t0, blk0 = max(pos0 - 3, 0) / kBlock8;
#pragma unroll
                for (int m = 0; m < 3; ++m) {
                    const int tm = t - 3 + m, pos = p.reverse ? L - 1 - tm : tm;
                    xh[m] *= sc[(pos / kBlock8 == blk0 ? 0 : H::G) + r.ch];
                }
            }
            if (t < 3)                                         // before the row: its history
#pragma unroll
                for (int m = 0; m < 3; ++m)
                    if (t - 3 + m < 0) xh[m] = past(r.ch, t - 3 + m);
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = prm[r.ch * 8 + k];
            auto tap = [&](int i, int lag) { return i >= lag ? u[i >= lag ? i - lag : 0] : xh[i >= lag ? 0 : 3 + i - lag]; };
            if (!p.since && p.conv_width == 4) {
#pragma unroll
                for (int i = 0; i < E; ++i)
#pragma unroll
                    for (int lag = 0; lag < 4; ++lag) acc[i] = fmaf(w[3 - lag], tap(i, lag), acc[i]);
            } else {                                           // an absent tap is no product with 0
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int sn = min(p.since ? since[r.tl + i] : 4, p.conv_width - 1);
#pragma unroll
                    for (int lag = 0; lag < 4; ++lag)
                        if (lag <= sn) acc[i] = fmaf(w[3 - lag], tap(i, lag), acc[i]);
                }
            }
        }
        each_pair(u, acc, [](uint64_t v) { return silu2(v); });
    }
    take<T, S, CL, Q8>(p, raw, 1, r, t0, dt);
    if constexpr (ADJ) {
        take<T, S, CL, Q8>(p, raw, 3, r, t0, g);
        if (p.z.p) {
            float z[E];
            take<T, S, CL, Q8>(p, raw, 2, r, t0, z);
            each_pair(z, z, [](uint64_t v) { return silu2(v); });
#pragma unroll
            for (int i = 0; i < E; ++i) g[i] *= z[i];
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) dt[i] += prm[r.c(i) * 8 + 5];
    // past 20 the softplus is its argument to fp32 by itself
    if (p.softplus) each_pair(dt, dt, [](uint64_t v) { return softplus2(v); });
#pragma unroll
    for (int i = 0; i < E; ++i) {
        float dl = dt[i];
        if (i >= hi) {
            dl = u[i] = 0.f;
            if (ADJ) g[i] = 0.f;
        }
        const int o = r.c(i) * (H::TT + 1) + r.t(i);
        const float du = dl * u[i];
        st[o] = make_float2(dl, du);
        if constexpr (HEADS) as[o] = expf(dl * prm[r.c(i) * 8 + 7]);
        if constexpr (ADJ) {
            gs[o] = g[i];
            us[r.c(i) * H::RO + r.t(i)] = u[i];
        }
    }
    if (tid < 32) {
        const uint32_t m = __ballot_sync(0xffffffffu, p.since && tid < H::TT && t0 + tid < L &&
                                                          since[tid < H::TT ? tid : 0] == 0);
        if (tid == 0) *mask = m;
    }
    // rows of B and C: the 4 states of a lane at a step, once per order
#pragma unroll
    for (int k = tid; k < S * H::TT * (ADJ ? 2 : 1); k += H::NH) {
        const int jj = k % S, tl = k / S % H::TT;
        const bool isC = ADJ && k >= S * H::TT;
        const T* src = reinterpret_cast<const T*>(raw + (isC ? R::C : R::B));
        float v[4];
        if constexpr (CL) {
            take_run<T, 4>(src + tl * (R::kBRow / R::ES) + 4 * jj, false, v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = Elem<T>::to_f(src[(4 * jj + i) * H::TT + (p.reverse ? H::TT - 1 - tl : tl)]);
        }
        float* dst = (isC ? Cs : Bs) + tl * H::RB + 4 * jj;
#pragma unroll
        for (int q = 0; q < H::NC; ++q)
            *reinterpret_cast<float4*>(dst + q * H::RQ) = make_float4(v[q], v[1 ^ q], v[2 ^ q], v[3 ^ q]);
    }
}

// A of one lane's 4 states (times log2 e), zeros past dim. Past d_state stands the last state's:
// those states hold zeros and keep them, as long as that state's decay is finite (a negative delta
// makes it grow), and the lane's smallest A is one of the channel's (see decays).
template <int S>
__device__ __forceinline__ void load_A(const BwdParams& p, int d, int j, uint64_t (&A2)[2]) {
    float a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int n = 4 * j + (k ^ slot_order<S>(d));
        a[k] = d < p.dim ? kLog2e * p.A[(int64_t)d * p.dstate + min(n, p.dstate - 1)] : 0.f;
    }
    A2[0] = pk2(a[0], a[1]);
    A2[1] = pk2(a[2], a[3]);
}

// Decays of T steps for a lane's 4 states, 2^(delta A log2 e), and the steps' delta u, from row.
// With A per head the decays are staged (from as).
// The SFU's exp comes out low on average: by 6e-9 of its value for exponents above -0.004, by 2e-8
// to 3e-8 from there to -1 (means over 0.5 M random arguments in each of 46 ranges). A state that
// decays by 1 - a per step collects such a bias over 1 / (1 - a) steps, which shows in dA. The
// exponent is therefore raised by that (over ln 2), in the multiply that forms it: by the one or the
// other for all T steps, as the first step's delta and the lane's smallest A say (1 % of the
// call's time). dA against fp64 over 4000 steps, in 1e-7 of its norm, at deltas of 2e-4 to 1e-3 /
// 1e-3 to 0.01 / 0.01 to 0.1: 22 / 12 / 4; torch's fp32 376 / 137 / 3; one raise for all, by 2.5e-8,
// 296 / 104 / 5, by 1.2e-8 70 / 29 / 11. An exponent of 0 (delta = 0) still gives 1 exactly: 6e-9 is
// far below half a step of it.
constexpr float kExpBiasSlow = 0.9e-8f, kExpBiasFast = 3.1e-8f, kSlow = 0.004f;
template <bool HEADS, int T>
__device__ __forceinline__ void decays(const uint64_t (&A2)[2], const float2* row, const float* as,
                                       uint64_t (&a)[T][2], uint64_t (&du2)[T]) {
    uint64_t raise = 0;
    if constexpr (!HEADS) {
        const float2 x = upk2(A2[0]), y = upk2(A2[1]);
        const float least = fminf(fminf(fabsf(x.x), fabsf(x.y)), fminf(fabsf(y.x), fabsf(y.y)));
        const float r = row[0].x * least < kSlow ? kExpBiasSlow : kExpBiasFast;
        raise = pk2(r, r);
    }
#pragma unroll
    for (int i = 0; i < T; ++i) {
        const float2 s = row[i];
        if constexpr (HEADS) {
            a[i][0] = a[i][1] = pk2(as[i], as[i]);
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 e = upk2(fma2(pk2(s.x, s.x), A2[k], raise));
                a[i][k] = pk2(ex2(e.x), ex2(e.y));
            }
        }
        du2[i] = pk2(s.y, s.y);
    }
}

// The sequence starts among the T steps of a sub-tile, bit i for step i. Nothing passes a start
// in either direction, not even a NaN, so zero decays would not do: a sub-tile that holds a
// start is worked out with a test at each step, all others without one.
template <int T> __device__ __forceinline__ uint32_t starts_in(uint32_t mask, int sub) {
    return mask >> (sub * T) & ((1u << T) - 1);
}
// A segment's product of decays that holds a start: no product of decays, which are not
// negative, comes out as this.
constexpr float kCut = -0.f;
__device__ __forceinline__ bool is_cut(float product) { return __float_as_uint(product) == 0x80000000u; }

__device__ __forceinline__ void ldpair(const float* s, uint64_t (&v)[2]) {
    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(s);
    v[0] = q.x;
    v[1] = q.y;
}
__device__ __forceinline__ void stpair(float* s, const uint64_t (&v)[2]) {
    *reinterpret_cast<ulonglong2*>(s) = make_ulonglong2(v[0], v[1]);
}

// A lane's states of a (batch, dim, dstate) tensor, zeros past dim or d_state or when null.
template <int S>
__device__ __forceinline__ void load_state(const BwdParams& p, const float* s, int b, int d, int j,
                                           uint64_t (&v)[2]) {
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int n = 4 * j + (k ^ slot_order<S>(d));
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

// The arrays of a staged tile (one of two).
template <int S> struct BwdStaged {
    using H = BwdShape<S>;
    float2* st;
    float *as, *gs, *us, *Bs, *Cs;
    __device__ __forceinline__ BwdStaged(float* sm, bool adj, bool heads) {
        st = reinterpret_cast<float2*>(sm);
        as = sm + H::kSt;
        gs = as + (heads ? H::kDecay : 0);
        us = gs + (adj ? H::kG : 0);
        Bs = us + (adj ? H::kU : 0);
        Cs = Bs + H::kBC;
    }
    __device__ __forceinline__ BwdStaged at(int n, int size) const {
        BwdStaged r = *this;
        r.st += n * size / 2;
        r.as += n * size;
        r.gs += n * size;
        r.us += n * size;
        r.Bs += n * size;
        r.Cs += n * size;
        return r;
    }
};

// The forward pass: checkpoints of the state (MODE kCheckpoint), or a segment's summary.
template <typename T, int S, bool CL, bool Q8, bool HEADS, int MODE>
__global__ void __launch_bounds__(BwdShape<S>::NT) scan_bwd_states_kernel(const BwdParams p) {
    using H = BwdShape<S>;
    constexpr bool SUM = MODE == kSummary;
    constexpr int KL = H::KL, ST = H::T;
    extern __shared__ __align__(16) float sm[];
    constexpr int kStaged = H::kStaged(SUM, HEADS);
    const BwdStaged<S> staged(sm, SUM, HEADS);
    float* prm = sm + 2 * kStaged;
    uint32_t* mask = reinterpret_cast<uint32_t*>(prm + H::kPrm);
    uint8_t* raw = reinterpret_cast<uint8_t*>(prm + H::kPrm + H::kMask);
    constexpr int kRaw = BwdRaw<T, S, CL>::bytes(Q8);
    using K = BwdCopies<T, S, CL, Q8, SUM>;
    BwdCopy* table = reinterpret_cast<BwdCopy*>(raw + 2 * kRaw);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int j = lane % S, cl = lane / S;
    const int b = blockIdx.y, d0 = blockIdx.x * H::G, seg = blockIdx.z;
    const int tb = seg * p.seg_len, te = min(p.seqlen, tb + p.seg_len);
    const int64_t row = (int64_t)seg * p.batch + b;
    load_prm<S>(p, d0, prm);
    __syncthreads();
    const int ntiles = (te - tb + H::TT - 1) / H::TT;

    if (warp >= H::W) {                                        // helper: tile n + 1 while n is scanned
        const int hid = tid - 32 * H::W;
        auto fetch = [&](int n) {
            fetch_tile<T, S, CL, Q8, SUM>(p, table, hid, b, d0, tb + n * H::TT, raw + (n & 1) * kRaw);
        };
        auto stage = [&](int n) {
            const BwdStaged<S> to = staged.at(n & 1, kStaged);
            stage_tile<T, S, CL, Q8, SUM, HEADS>(p, hid, b, d0, tb + n * H::TT, raw + (n & 1) * kRaw, prm, to.st, to.as, to.gs,
                                          to.us, to.Bs, to.Cs, mask + (n & 1));
        };
        if (p.async)                                           // a thread reads back its own entries
            for (int k = hid; k < K::COUNT; k += H::NH) table[k] = K::make(p, b, d0, k);
        fetch(0);
        for (int n = -1; n < ntiles; ++n) {
            cp_async_wait();
            named_bar_sync(1, H::NH);                          // tile n + 1 is here, n has been staged
            if (n + 2 < ntiles) fetch(n + 2);
            if (n + 1 < ntiles) stage(n + 1);
            __syncthreads();
        }
        return;
    }

    uint64_t h[H::KC][KL][2], A2[H::KC][KL][2], R[H::KC][KL][2], P[H::KC][KL][2];
#pragma unroll
    for (int kc = 0; kc < H::KC; ++kc)
#pragma unroll
        for (int kl = 0; kl < KL; ++kl) {
            const int d = d0 + H::channel(warp, kc, cl, j, kl);
            if constexpr (!HEADS) load_A<S>(p, d, j, A2[kc][kl]);
            R[kc][kl][0] = R[kc][kl][1] = 0;
            P[kc][kl][0] = P[kc][kl][1] = pk2(1.f, 1.f);
            h[kc][kl][0] = h[kc][kl][1] = 0;
            if (!SUM && seg == 0) load_state<S>(p, p.h0, b, d, j, h[kc][kl]);
            if (!SUM && seg > 0 && d < p.dim) ldpair(p.sumS + ns_off<S>(p, row, d, j), h[kc][kl]);
        }
    __syncthreads();                                           // tile 0 is staged
    bool alive = true;                                         // no start in the segment so far
    for (int n = 0; n < ntiles; ++n) {
        const int t0 = tb + n * H::TT;
        const BwdStaged<S> in = staged.at(n & 1, kStaged);
        const uint32_t starts = HEADS ? 0 : mask[n & 1];       // (not with A per head)
#pragma unroll
        for (int kc = 0; kc < H::KC; ++kc) {
            const int q = slot_order<S>(H::channel(warp, kc, cl, 0, 0));
#pragma unroll 1
            for (int sub = 0; sub < H::NSUB; ++sub) {
                const float* Br = in.Bs + q * H::RQ + sub * ST * H::RB + 4 * j;
                const float* Cr = in.Cs + q * H::RQ + sub * ST * H::RB + 4 * j;
                uint64_t a[KL][ST][2], du2[KL][ST];
                int so[KL];
#pragma unroll
                for (int kl = 0; kl < KL; ++kl) {
                    const int c = H::channel(warp, kc, cl, j, kl);
                    so[kl] = c * (H::TT + 1) + sub * ST;
                    if (!SUM && d0 + c < p.dim)
                        stpair(p.ckpt + ns_off<S>(p, (int64_t)b * p.nsub + t0 / ST + sub, d0 + c, j), h[kc][kl]);
                    decays<HEADS, ST>(A2[kc][kl], in.st + so[kl], in.as + so[kl], a[kl], du2[kl]);
                }
                const uint32_t cuts = starts_in<ST>(starts, sub);
                bool on = alive && (starts & ((1u << sub * ST) - 1)) == 0;
                auto steps = [&](auto cutting, auto summing) {
                    constexpr bool CUT = decltype(cutting)::value, ADD = decltype(summing)::value;
#pragma unroll
                    for (int i = 0; i < ST; ++i) {
                        if (CUT && (cuts >> i & 1)) {
                            on = false;
#pragma unroll
                            for (int kl = 0; kl < KL; ++kl) {
                                h[kc][kl][0] = h[kc][kl][1] = 0;
                                P[kc][kl][0] = P[kc][kl][1] = pk2(kCut, kCut);
                            }
                        }
                        uint64_t bv[2], cv[2];
                        ldpair(Br + i * H::RB, bv);
                        if (ADD) ldpair(Cr + i * H::RB, cv);
#pragma unroll
                        for (int kl = 0; kl < KL; ++kl) {
                            uint64_t g2 = 0;
                            if (ADD) g2 = pk2(in.gs[so[kl] + i], in.gs[so[kl] + i]);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                h[kc][kl][k] = fma2(a[kl][i][k], h[kc][kl][k], mul2(du2[kl][i], bv[k]));
                                if (ADD && (!CUT || on)) {
                                    P[kc][kl][k] = mul2(P[kc][kl][k], a[kl][i][k]);
                                    R[kc][kl][k] = fma2(P[kc][kl][k], mul2(g2, cv[k]), R[kc][kl][k]);
                                }
                            }
                        }
                    }
                };
                std::bool_constant<SUM> sums;
                if constexpr (HEADS) {
                    steps(std::false_type{}, sums);
                } else {
                    if (cuts) steps(std::true_type{}, sums);
                    else if (SUM && !on) steps(std::false_type{}, std::false_type{});
                    else steps(std::false_type{}, sums);
                }
            }
        }
        alive = alive && starts == 0;
        __syncthreads();                                       // tile n is done, n + 1 staged
    }
    if (SUM) {
#pragma unroll
        for (int kc = 0; kc < H::KC; ++kc)
#pragma unroll
            for (int kl = 0; kl < KL; ++kl) {
                const int d = d0 + H::channel(warp, kc, cl, j, kl);
                if (d < p.dim) {
                    const int64_t o = ns_off<S>(p, row, d, j);
                    stpair(p.sumP + o, P[kc][kl]);
                    stpair(p.sumS + o, h[kc][kl]);
                    stpair(p.sumR + o, R[kc][kl]);
                }
            }
    }
}

// Chains the segments' summaries: sumS[seg] becomes the state before the segment, sumR[seg]
// the adjoint carry a_t lam_t from behind it. One thread per (batch row, channel, state).
template <int S>
__global__ void __launch_bounds__(256) scan_bwd_carry_kernel(const BwdParams p) {
    constexpr int NS = 4 * S, U = 8;                           // U segments' loads together
    const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t per = (int64_t)p.batch * p.dim * NS;
    if (idx >= per) return;
    const uint32_t bd = (uint32_t)(idx / NS);                  // batch * dim is below 2^31
    const int n = (int)(idx % NS) ^ slot_order<S>((int)(bd % (uint32_t)p.dim));
    float h = p.h0 && n < p.dstate ? p.h0[(int64_t)bd * p.dstate + n] : 0.f;
    float m = p.dhl && n < p.dstate ? p.dhl[(int64_t)bd * p.dstate + n] : 0.f;
    const float* P = p.sumP + idx;
    float *Sx = p.sumS + idx, *Rx = p.sumR + idx;
    for (int s0 = 0; s0 < p.nseg; s0 += U) {
        float pr[U], e[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s0 + k < p.nseg) {
                pr[k] = P[(s0 + k) * per];
                e[k] = Sx[(s0 + k) * per];
            }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s0 + k < p.nseg) {
                Sx[(s0 + k) * per] = h;
                h = is_cut(pr[k]) ? e[k] : fmaf(pr[k], h, e[k]);
            }
    }
    for (int s0 = p.nseg - 1; s0 >= 0; s0 -= U) {
        float pr[U], r[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s0 - k >= 0) {
                pr[k] = P[(s0 - k) * per];
                r[k] = Rx[(s0 - k) * per];
            }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s0 - k >= 0) {
                Rx[(s0 - k) * per] = m;
                m = is_cut(pr[k]) ? r[k] : fmaf(pr[k], m, r[k]);
            }
    }
}

// The backward sweep.
template <typename T, int S, bool CL, bool Q8, bool HEADS>
__global__ void __launch_bounds__(BwdShape<S>::NT, BwdSmem<T, S, CL, Q8, HEADS>::CTAS)
scan_bwd_kernel(const BwdParams p) {
    using H = BwdShape<S>;
    constexpr int KC = H::KC, KL = H::KL, ST = H::T, TT = H::TT, E = H::EPT;
    constexpr bool REGS = KC == 1;                             // m and dA in registers, else carried over
    extern __shared__ __align__(16) float sm[];
    constexpr int kStaged = H::kStaged(true, HEADS);
    const BwdStaged<S> staged(sm, true, HEADS);
    float* outs = sm + 2 * kStaged;                            // y, s1, s2 of two tiles
    float* part = outs + 6 * H::kOut;
    float* prm = part + H::kPart;
    uint32_t* mask = reinterpret_cast<uint32_t*>(prm + H::kPrm);
    float* carry = prm + H::kPrm + H::kMask;
    float* sums = carry + H::kCarry;
    uint8_t* raw = reinterpret_cast<uint8_t*>(sums + (CL ? H::kSum : 0));
    constexpr int kRaw = BwdRaw<T, S, CL>::bytes(Q8);
    using K = BwdCopies<T, S, CL, Q8, true>;
    BwdCopy* table = reinterpret_cast<BwdCopy*>(raw + 3 * kRaw);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int j = lane % S, cl = lane / S;
    const int b = blockIdx.y, d0 = blockIdx.x * H::G, seg = blockIdx.z;
    const int L = p.seqlen, tb = seg * p.seg_len, te = min(L, tb + p.seg_len);
    const int64_t row = (int64_t)seg * p.batch + b;
    load_prm<S>(p, d0, prm);

    const int ntiles = (te - tb + TT - 1) / TT;
    __syncthreads();

    if (warp >= H::W) {
        // Helper. While tile n (counted from the segment's end) is scanned: the gradients of
        // tile n - 1, then tile n + 1 into the staged tile that n - 1 leaves.
        const int hid = tid - 32 * H::W;
        const BwdRun<S, CL> run(hid);
        LongSum dD, dBias;                                     // rows: of the run's channel; CL: of channel hid
        if constexpr (CL) {
            for (int k = hid; k < H::kSum; k += H::NH) sums[k] = 0.f;
        }
        // channel-last: the sums of a tile's places, one thread a channel
        auto drain = [&] {
            static_assert(H::G <= H::NH, "a thread per channel");
            named_bar_sync(1, H::NH);
            if (hid < H::G) {
                float v0 = 0.f, v1 = 0.f;
                for (int t = 0; t < TT; ++t) {
                    float *a = sums + hid * TT + t, *b = a + H::G * TT;
                    v0 += *a;
                    v1 += *b;
                    *a = *b = 0.f;
                }
                dD.add(v0);
                dBias.add(v1);
            }
            named_bar_sync(1, H::NH);
        };
        auto start = [&](int n) { return tb + (ntiles - 1 - n) * TT; };
        auto fetch = [&](int n) {
            fetch_tile<T, S, CL, Q8, true>(p, table, hid, b, d0, start(n), raw + n % 3 * kRaw);
        };
        auto stage = [&](int n) {
            const BwdStaged<S> to = staged.at(n & 1, kStaged);
            stage_tile<T, S, CL, Q8, true, HEADS>(p, hid, b, d0, start(n), raw + n % 3 * kRaw, prm, to.st, to.as, to.gs, to.us,
                                           to.Bs, to.Cs, mask + (n & 1));
        };
        // the gradients of a tile, one run per thread
        auto finish = [&](int n) {
            const int t0 = start(n);
            const BwdStaged<S> in = staged.at(n & 1, kStaged);
            const uint8_t* from = raw + n % 3 * kRaw;
            const float* ys = outs + (n & 1) * 3 * H::kOut;
            const float *s1s = ys + H::kOut, *s2s = s1s + H::kOut;
            const int d = d0 + run.ch, t = t0 + run.tl;
            const int pos = p.reverse ? L - 1 - t : t;
            const int hi = CL ? (t < L ? min(E, p.dim - d) : 0) : (d < p.dim ? min(E, L - t) : 0);
            if (hi > 0) {
                float dt[E], z[E], dy[E], du[E], ddt[E], dz[E], tileD = 0.f, tileBias = 0.f;
                take<T, S, CL, Q8>(p, from, 1, run, t0, dt);
                if (p.z.p) {
                    take<T, S, CL, Q8>(p, from, 2, run, t0, z);
                    take<T, S, CL, Q8>(p, from, 3, run, t0, dy);
                }
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int c = run.c(i), tl = run.t(i), o = c * H::RO + tl;
                    const float2 s = in.st[c * (TT + 1) + tl];
                    const float g = in.gs[c * (TT + 1) + tl];
                    const float u = in.us[o], Dv = prm[c * 8 + 6];
                    const float s1 = s1s[o], s2 = s2s[o] * (HEADS ? prm[c * 8 + 7] : kLn2);
                    du[i] = fmaf(g, Dv, s.x * s1);
                    const float ddelta = fmaf(u, s1, s2);
                    ddt[i] = p.softplus ? ddelta * sigmoidf_(dt[i] + prm[c * 8 + 5]) : ddelta;
                    if (p.z.p) {
                        const float sg = sigmoidf_(z[i]);
                        dz[i] = dy[i] * fmaf(Dv, u, ys[o]) * (sg * fmaf(z[i], 1.f - sg, 1.f));
                    }
                    if (CL) {
                        if (i < hi) {
                            sums[c * TT + tl] += g * u;
                            sums[H::G * TT + c * TT + tl] += ddt[i];
                        }
                    } else if (i < hi) {
                        tileD = fmaf(g, u, tileD);             // the run first: fewer roundings of
                        tileBias += ddt[i];                    // the long sum
                    }
                }
                if constexpr (!CL) {
                    dD.add(tileD);
                    dBias.add(tileBias);
                }
                if constexpr (CL) {
                    auto at = [&](const Str& s) { return (int64_t)b * s.b + d + (int64_t)pos * s.p; };
                    if (p.du32) put_run<float, E>(p.du32 + at(p.sdu), false, p.vec_out, hi, du);
                    else put_run<T, E>(static_cast<T*>(p.du) + at(p.sdu), false, p.vec_out, hi, du);
                    put_run<T, E>(static_cast<T*>(p.ddt) + at(p.sddt), false, p.vec_out, hi, ddt);
                    if (p.z.p && p.dz)
                        put_run<T, E>(static_cast<T*>(p.dz) + at(p.sdz), false, p.vec_out, hi, dz);
                } else {
                    // dense rows: one offset for all, of the run's lowest position
                    const bool rev = p.reverse;
                    const int64_t at = ((int64_t)b * p.dim + d) * L + (rev ? pos - (E - 1) : pos);
                    if (p.du32) put_run<float, E>(p.du32 + at, rev, p.vec_out, hi, du);
                    else put_run<T, E>(static_cast<T*>(p.du) + at, rev, p.vec_out, hi, du);
                    put_run<T, E>(static_cast<T*>(p.ddt) + at, rev, p.vec_out, hi, ddt);
                    if (p.z.p && p.dz) put_run<T, E>(static_cast<T*>(p.dz) + at, rev, p.vec_out, hi, dz);
                }
            }
        };
        if (p.async)                                           // a thread reads back its own entries
            for (int k = hid; k < K::COUNT; k += H::NH) table[k] = K::make(p, b, d0, k);
        fetch(0);
        for (int n = -1; n < ntiles; ++n) {
            cp_async_wait();
            if (n > 0) finish(n - 1);
            if (CL && n > 0 && n % H::DRAIN == 0) drain();
            named_bar_sync(1, H::NH);                          // tile n + 1 is here, n - 1 finished
            if (n + 2 < ntiles) fetch(n + 2);
            if (n + 1 < ntiles) stage(n + 1);
            __syncthreads();
        }
        finish(ntiles - 1);
        if constexpr (!CL) {
            // the threads of a channel are neighbours within a warp (TT / EPT of them)
            constexpr int PER = TT / E;
            float v0 = dD.get(), v1 = dBias.get();
#pragma unroll
            for (int w = 1; w < PER; w *= 2) {
                v0 += __shfl_xor_sync(0xffffffffu, v0, w);
                v1 += __shfl_xor_sync(0xffffffffu, v1, w);
            }
            if (hid % PER == 0 && d0 + run.ch < p.dim) {
                float* o = p.pD + (row * p.dim + d0 + run.ch) * 2;
                o[0] = v0;
                o[1] = v1;
            }
        } else {
            drain();
            if (hid < H::G && d0 + hid < p.dim) {
                float* o = p.pD + (row * p.dim + d0 + hid) * 2;
                o[0] = dD.get();
                o[1] = dBias.get();
            }
        }
        return;
    }

    uint64_t m[KL][2], dA[KL][2], A2[KL][2];
    // where a thread keeps them between its groups of channels
    auto place = [&](int kc, int kl) { return carry + ((size_t)(kc * KL + kl) * 32 * H::W + tid) * 8; };
#pragma unroll
    for (int kc = 0; kc < KC; ++kc)
#pragma unroll
        for (int kl = 0; kl < KL; ++kl) {
            const int d = d0 + H::channel(warp, kc, cl, j, kl);
            dA[kl][0] = dA[kl][1] = 0;
            m[kl][0] = m[kl][1] = 0;
            if (te == L) load_state<S>(p, p.dhl, b, d, j, m[kl]);
            else if (d < p.dim) ldpair(p.sumR + ns_off<S>(p, row, d, j), m[kl]);
            if constexpr (REGS) {
                if constexpr (!HEADS) load_A<S>(p, d, j, A2[kl]);
            } else {
                stpair(place(kc, kl), m[kl]);
                stpair(place(kc, kl) + 4, dA[kl]);
            }
        }
    // The states before the next sub-tile to come (from the segment's last one backwards), for
    // group kc: fetched one use ahead.
    const float* ck = p.ckpt + ns_off<S>(p, (int64_t)b * p.nsub + (tb + (ntiles - 1) * TT) / ST + H::NSUB - 1, d0, j);
    const int64_t ck_step = (int64_t)p.dim * H::NS;
    uint64_t hn[KL][2];
    auto load_ckpt = [&](int kc) {
#pragma unroll
        for (int kl = 0; kl < KL; ++kl) {
            const int c = H::channel(warp, kc, cl, j, kl);
            if (d0 + c < p.dim) ldpair(ck + c * H::NS, hn[kl]);
        }
    };
#pragma unroll
    for (int kl = 0; kl < KL; ++kl) hn[kl][0] = hn[kl][1] = 0;
    load_ckpt(0);
    int left = ntiles * H::NSUB;                               // sub-tiles to come
    // dA of the steps since the last call: added to the long sums in scratch memory (every DRAIN
    // tiles), or (last) the whole sum left there. A thread comes back to the places it wrote.
    auto drain = [&](bool first, bool last) {
        auto put = [&](int64_t o, float v) {
            LongSum s;
            if (!first) {
                s.hi = p.pA[o];
                s.lo = p.pA_lo[o];
            }
            s.add(v);
            p.pA[o] = last ? s.get() : s.hi;
            if (!last) p.pA_lo[o] = s.lo;
        };
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
#pragma unroll
            for (int kl = 0; kl < KL; ++kl) {
                const int d = d0 + H::channel(warp, kc, cl, j, kl);
                if constexpr (!REGS) ldpair(place(kc, kl) + 4, dA[kl]);
                if (!HEADS && d < p.dim) {
                    const int64_t o = ns_off<S>(p, row, d, j);
                    if (first && last) {
                        stpair(p.pA + o, dA[kl]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 f = upk2(dA[kl][k]);
                            put(o + 2 * k, f.x);
                            put(o + 2 * k + 1, f.y);
                        }
                    }
                }
            }
            if constexpr (HEADS) {                             // (rows, dim): summed over the states
                constexpr bool kTrade = StateSums<S>::kTrade;
                float v[KL];
#pragma unroll
                for (int kl = 0; kl < KL; ++kl) {
                    const float2 f = upk2(add2(dA[kl][0], dA[kl][1]));
                    v[kl] = f.x + f.y;
                }
                if constexpr (kTrade) v[0] += __shfl_xor_sync(0xffffffffu, v[KL - 1], 1);
#pragma unroll
                for (int w = kTrade ? 2 : 1; w < S; w *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
                const int d = d0 + H::channel(warp, kc, cl, j, 0);
                if (j < (kTrade ? 2 : 1) && d < p.dim) put(row * p.dim + d, v[0]);
            }
#pragma unroll
            for (int kl = 0; kl < KL; ++kl) {
                dA[kl][0] = dA[kl][1] = 0;
                if constexpr (!REGS) stpair(place(kc, kl) + 4, dA[kl]);
            }
        }
    };
    // the CTA's dB and dC of the PS steps from t on: the sum over its warps
    auto flush = [&](int t) {
        constexpr int ROW = 2 * H::NS, PS = H::PS;
        named_bar_sync(2, 32 * H::W);
        float* out = p.parts + (((int64_t)blockIdx.x * p.batch + b) * L + t) * ROW;
        const int n = min(PS, te - t) * ROW;                   // below 1 past the segment's end
#pragma unroll
        for (int k = tid * 4; k < PS * ROW; k += 32 * H::W * 4) {
            if (k >= n) break;
            const float* from = part + k / ROW * H::RP + k % ROW;
            float4 v = *reinterpret_cast<const float4*>(from);
#pragma unroll
            for (int w = 1; w < H::W; ++w) {
                const float4 q = *reinterpret_cast<const float4*>(from + w * PS * H::RP);
                v.x += q.x;
                v.y += q.y;
                v.z += q.z;
                v.w += q.w;
            }
            *reinterpret_cast<float4*>(out + k) = v;
        }
        if (PS < TT) named_bar_sync(2, 32 * H::W);
    };
    __syncthreads();                                           // tile 0 is staged
    for (int n = 0; n < ntiles; ++n) {
        const int tile = ntiles - 1 - n, t0 = tb + tile * TT;
        const BwdStaged<S> in = staged.at(n & 1, kStaged);
        const float2* st = in.st;
        const float* gs = in.gs;
        const float *Bs = in.Bs, *Cs = in.Cs;
        float* ys = outs + (n & 1) * 3 * H::kOut;
        float *s1s = ys + H::kOut, *s2s = s1s + H::kOut;
        const uint32_t starts = HEADS ? 0 : mask[n & 1];
#pragma unroll 1
        for (int sub = H::NSUB - 1; sub >= 0; --sub) {
            constexpr int PT = 4 / H::NC;                      // dB, dC values left per step
            float rB[ST * PT], rC[ST * PT];
            if constexpr (KC > 1) {
#pragma unroll
                for (int i = 0; i < ST * PT; ++i) rB[i] = rC[i] = 0.f;
            }
#pragma unroll 1
            for (int kc = 0; kc < KC; ++kc) {
                const int sq = slot_order<S>(H::channel(warp, kc, cl, 0, 0));
                uint64_t h0[KL][2];
#pragma unroll
                for (int kl = 0; kl < KL; ++kl) {
                    h0[kl][0] = hn[kl][0];
                    h0[kl][1] = hn[kl][1];
                }
                if (kc + 1 < KC) {
                    load_ckpt(kc + 1);
                } else if (--left > 0) {
                    ck -= ck_step;
                    load_ckpt(0);
                }
                int so[KL];
#pragma unroll
                for (int kl = 0; kl < KL; ++kl) {
                    const int c = H::channel(warp, kc, cl, j, kl);
                    so[kl] = c * (TT + 1) + sub * ST;
                    if constexpr (!REGS) {
                        if constexpr (!HEADS) load_A<S>(p, d0 + c, j, A2[kl]);
                        ldpair(place(kc, kl), m[kl]);
                        ldpair(place(kc, kl) + 4, dA[kl]);
                    }
                }
                const float* Br = Bs + sq * H::RQ + sub * ST * H::RB + 4 * j;
                const float* Cr = Cs + sq * H::RQ + sub * ST * H::RB + 4 * j;
                const uint32_t cuts = starts_in<ST>(starts, sub);
                float y[8], s1[8], s2[8];
                auto steps = [&](auto cutting) {
                    constexpr bool CUT = decltype(cutting)::value;
                    uint64_t a[KL][ST][2], h[KL][ST][2];
                    {
                        uint64_t du2[KL][ST];
#pragma unroll
                        for (int kl = 0; kl < KL; ++kl)
                            decays<HEADS, ST>(A2[kl], st + so[kl], in.as + so[kl], a[kl], du2[kl]);
#pragma unroll
                        for (int i = 0; i < ST; ++i) {
                            uint64_t bv[2];
                            ldpair(Br + i * H::RB, bv);
#pragma unroll
                            for (int kl = 0; kl < KL; ++kl)
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    uint64_t before = i ? h[kl][i ? i - 1 : 0][k] : h0[kl][k];
                                    if (CUT && (cuts >> i & 1)) before = 0;
                                    h[kl][i][k] = fma2(a[kl][i][k], before, mul2(du2[kl][i], bv[k]));
                                }
                        }
                    }
#pragma unroll
                    for (int i = ST - 1; i >= 0; --i) {
                        uint64_t bv[2], cv[2], tb2[2], tc2[2];
                        ldpair(Br + i * H::RB, bv);
                        ldpair(Cr + i * H::RB, cv);
#pragma unroll
                        for (int kl = 0; kl < KL; ++kl) {
                            const float2 s = st[so[kl] + i];
                            const float g = gs[so[kl] + i];
                            const uint64_t d2 = pk2(s.x, s.x), du2 = pk2(s.y, s.y), g2 = pk2(g, g);
                            uint64_t lam[2], q[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                lam[k] = fma2(g2, cv[k], m[kl][k]);
                                m[kl][k] = mul2(a[kl][i][k], lam[k]);
                                q[k] = mul2(m[kl][k], i ? h[kl][i ? i - 1 : 0][k] : h0[kl][k]);
                                if (CUT && (cuts >> i & 1)) m[kl][k] = q[k] = 0;
                                dA[kl][k] = fma2(q[k], d2, dA[kl][k]);
                                tb2[k] = kl ? fma2(lam[k], du2, tb2[k]) : mul2(lam[k], du2);
                                tc2[k] = kl ? fma2(g2, h[kl][i][k], tc2[k]) : mul2(g2, h[kl][i][k]);
                            }
                            const int v = kl * ST + i;
                            const float2 fy = upk2(fma2(cv[1], h[kl][i][1], mul2(cv[0], h[kl][i][0])));
                            const float2 f1 = upk2(fma2(bv[1], lam[1], mul2(bv[0], lam[0])));
                            y[v] = fy.x + fy.y;
                            s1[v] = f1.x + f1.y;
                            if constexpr (HEADS) {
                                const float2 f2 = upk2(add2(q[0], q[1]));
                                s2[v] = f2.x + f2.y;                // times A: see finish()
                            } else {
                                const float2 f2 = upk2(fma2(q[1], A2[kl][1], mul2(q[0], A2[kl][0])));
                                s2[v] = f2.x + f2.y;
                            }
                        }
                        float vb[PT], vc[PT];
                        reduce_slots<S>(tb2, vb);
                        reduce_slots<S>(tc2, vc);
#pragma unroll
                        for (int k = 0; k < PT; ++k) {
                            rB[i * PT + k] = KC > 1 ? rB[i * PT + k] + vb[k] : vb[k];
                            rC[i * PT + k] = KC > 1 ? rC[i * PT + k] + vc[k] : vc[k];
                        }
                    }
                };
                if (!HEADS && cuts) steps(std::bool_constant<!HEADS>{});
                else steps(std::false_type{});
                using Sums = StateSums<S>;
                Sums::sum(y, lane);
                Sums::sum(s1, lane);
                Sums::sum(s2, lane);
                constexpr int SPAN = Sums::kTrade ? 2 * (ST / Sums::kept()) : ST / Sums::kept();
                if (j < SPAN) {                                // lanes beyond hold the same sums
                    const int c = H::channel(warp, kc, cl, j, 0);
                    const int o = c * H::RO + sub * ST + Sums::first(lane);
#pragma unroll
                    for (int k = 0; k < Sums::kept(); ++k) {
                        ys[o + k] = y[k];
                        s1s[o + k] = s1[k];
                        s2s[o + k] = s2[k];
                    }
                }
                if constexpr (!REGS) {
#pragma unroll
                    for (int kl = 0; kl < KL; ++kl) {
                        stpair(place(kc, kl), m[kl]);
                        stpair(place(kc, kl) + 4, dA[kl]);
                    }
                }
            }
            const int sq = slot_order<S>(H::channel(0, 0, cl, 0, 0));
            if constexpr (PT == 1) {
                using Sums = GroupSums<S>;
                Sums::sum(rB, lane);
                Sums::sum(rC, lane);
                const int first = Sums::first(lane);
#pragma unroll
                for (int k = 0; k < Sums::kept(); ++k) {
                    float* o = part + (warp * H::PS + (H::PS == TT ? sub * ST : 0) + first + k) * H::RP + 4 * j + sq;
                    o[0] = rB[k];
                    o[H::NS] = rC[k];
                }
            } else {
#pragma unroll
                for (int k = 0; k < ST * PT; ++k) {            // slot k % PT * NC of step k / PT
                    float* o = part + (warp * H::PS + (H::PS == TT ? sub * ST : 0) + k / PT) * H::RP + 4 * j +
                               (k % PT * H::NC ^ sq);
                    o[0] = rB[k];
                    o[H::NS] = rC[k];
                }
            }
            if constexpr (H::PS == ST) flush(t0 + sub * ST);   // the next sub-tile takes its place
        }
        if constexpr (H::PS == TT) flush(t0);
        if ((n + 1) % H::DRAIN == 0 && n + 1 < ntiles) drain(n + 1 == H::DRAIN, false);
        __syncthreads();                                       // tile n is done, n + 1 staged
    }
    // what the sweep summed over its steps
    drain(ntiles <= H::DRAIN, true);
    if (seg == 0 && p.dh0) {
#pragma unroll
        for (int kc = 0; kc < KC; ++kc)
#pragma unroll
            for (int kl = 0; kl < KL; ++kl) {
                const int d = d0 + H::channel(warp, kc, cl, j, kl);
                if constexpr (!REGS) ldpair(place(kc, kl), m[kl]);
                if (d >= p.dim) continue;
                const float2 lo = upk2(m[kl][0]), hi = upk2(m[kl][1]);
                const float f[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int n = 4 * j + (k ^ slot_order<S>(d));
                    if (n < p.dstate) p.dh0[((int64_t)b * p.dim + d) * p.dstate + n] = f[k];
                }
            }
    }
}

}  // namespace ssm
