// 8-bit kernels for sm_100a: activations packed for a backward pass, and the decode states'
// cache. A group (64 positions of a channel, or a channel's row of states) is held as int8
// codes round(127 x / max|x|) and one fp32 scale max|x| / 127. All are bound by memory:
// each value is read once and each code written once.
//
// Rounding. r = x * (127 / max) in fp32 is within 127 * 2^-23 of the quotient (two
// roundings of relative size 2^-24 each), so r decides the code unless it lies within
// 1e-4 of a border; there the quotient is taken again in fp64 (about one value in 5000):
// 127 x is exact and the division correctly rounded, so a quotient that is a tie comes out
// as one, and no other does (it is at least 2^-25 of its size away).
#pragma once

#include "device_common.cuh"
#include "quant_params.h"
#include "scan_bwd_kernel.cuh"

namespace ssm {

constexpr float kTiny8 = 7.888609052210118e-31f;               // 2^-100

// The bits of |x|, which order as the magnitudes do and put infinities and NaN on top.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

struct Quant {
    float top, inv, scale;
    __device__ __forceinline__ explicit Quant(uint32_t bits) {
        top = __uint_as_float(bits);
        const bool bad = bits >= 0x7f800000u, zero = top < kTiny8;
        inv = bad || zero ? 0.f : __fdiv_rn(127.f, top);
        scale = bad ? __uint_as_float(0x7fffffffu) : zero ? 0.f : __fdiv_rn(top, 127.f);
    }
    // round(127 x / top), ties to even
    __device__ __forceinline__ int nearest(float x) const {
        if (inv == 0.f) return 0;
        const float r = __fmul_rn(x, inv), q = rintf(r);
        if (fabsf(fabsf(r - q) - 0.5f) < 1e-4f)
            return (int)rint(__ddiv_rn(127.0 * (double)x, (double)top));
        return (int)q;
    }
    // floor(127 x / top + offset), the offset the top 24 bits of `bits` as a fraction
    __device__ __forceinline__ int dithered(float x, uint32_t bits) const {
        if (inv == 0.f) return 0;
        const float o = (float)(bits >> 8) * 0x1p-24f;
        const float t = __fadd_rn(__fmul_rn(x, inv), o);
        float q = floorf(t);
        if (fabsf(t - rintf(t)) < 1e-4f)
            q = (float)floor(__ddiv_rn(127.0 * (double)x, (double)top) + (double)o);
        return (int)fminf(q, 127.f);
    }
};

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}
__device__ __forceinline__ float code_at(uint32_t w, int k) { return (float)(int8_t)(w >> (8 * k)); }

// Eight codes of a run: one 8-byte access when aligned and whole, else byte by byte.
__device__ __forceinline__ void store_codes(int8_t* p, int hi, const int (&q)[8]) {
    if (hi >= 8 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < hi) p[i] = (int8_t)q[i];
}
__device__ __forceinline__ void load_codes(const int8_t* p, int hi, float (&f)[8]) {
    if (hi >= 8 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = code_at(i < 4 ? w.x : w.y, i % 4);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < hi ? (float)p[i] : 0.f;
}

// ------------------------------------------------------------------ activations --

// (batch, dim, seqlen): 8 neighbouring lanes hold a block of 64 positions.
template <typename T>
__global__ void __launch_bounds__(256) pack_row_kernel(const PackParams p) {
    const int nb = (p.seqlen + kBlock8 - 1) / kBlock8;
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x, blk = idx / 8;
    const int64_t rows = (int64_t)p.batch * p.dim;
    const bool in = blk < rows * nb;
    const int64_t row = in ? blk / nb : 0;
    const int t = in ? (int)(blk % nb) * kBlock8 + (int)(idx % 8) * 8 : p.seqlen;
    const int hi = min(8, p.seqlen - t);
    float x[8];
    load_run<T, 8>(static_cast<const T*>(p.x) + row * p.seqlen + t, 1, 0, hi, x);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, mag_bits(x[i]));
#pragma unroll
    for (int w = 1; w < 8; w *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, w));
    const Quant qz(top);
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = qz.nearest(x[i]);
    store_codes(p.codes + row * p.seqlen + t, hi, q);
    if (in && idx % 8 == 0) p.scales[blk] = qz.scale;
}

// Channel-last: a warp takes 8 positions of 256 channels (8 a lane), a CTA of 8 warps one
// block of 64 positions; the warps' maxima meet in shared memory.
template <typename T>
__global__ void __launch_bounds__(256) pack_cl_kernel(const PackParams p) {
    __shared__ uint32_t tops[8][256];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int d = blockIdx.x * 256 + lane * 8, b = blockIdx.z;
    const int nb = (p.seqlen + kBlock8 - 1) / kBlock8;
    const int hi = min(8, p.dim - d);
    for (int blk = blockIdx.y; blk < nb; blk += gridDim.y) {
        const int t0 = blk * kBlock8 + warp * 8;
        float x[8][8];
        uint32_t top[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int t = t0 + r;
            load_run<T, 8>(static_cast<const T*>(p.x) + ((int64_t)b * p.seqlen + t) * p.sx + d, 1, 0,
                           t < p.seqlen ? hi : 0, x[r]);
#pragma unroll
            for (int i = 0; i < 8; ++i) top[i] = max(top[i], mag_bits(x[r][i]));
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) tops[warp][i * 32 + lane] = top[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int w = 0; w < 8; ++w) top[i] = max(top[i], tops[w][i * 32 + lane]);
            const Quant qz(top[i]);
#pragma unroll
            for (int r = 0; r < 8; ++r) x[r][i] = (float)qz.nearest(x[r][i]);
            if (warp == 0 && i < hi) p.scales[((int64_t)b * nb + blk) * p.dim + d + i] = qz.scale;
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            int q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = (int)x[r][i];
            if (t0 + r < p.seqlen)
                store_codes(p.codes + ((int64_t)b * p.seqlen + t0 + r) * p.dim + d, hi, q);
        }
    }
}

// A thread reads 8 values back, along the positions of a channel or along the channels.
template <typename T, bool CL>
__global__ void __launch_bounds__(256) unpack_kernel(const PackParams p) {
    const int inner = CL ? p.dim : p.seqlen, runs = (inner + 7) / 8;
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x, row = idx / runs;
    const int nb = (p.seqlen + kBlock8 - 1) / kBlock8;
    if (row >= (int64_t)p.batch * (CL ? p.seqlen : p.dim)) return;
    const int k = (int)(idx % runs) * 8, hi = min(8, inner - k);
    float f[8];
    load_codes(p.codes + row * inner + k, hi, f);
    if constexpr (CL) {
        const int64_t b = row / p.seqlen;
        const int blk = (int)(row % p.seqlen) / kBlock8;
        float s[8];
        load_run<float, 8>(p.scales + (b * nb + blk) * p.dim + k, 1, 0, hi, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= s[i];
    } else {
        const float s = p.scales[row * nb + k / kBlock8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= s;
    }
    store_run<T, 8>(static_cast<T*>(p.out) + row * inner + k, 1, 0, hi, f);
}

// ----------------------------------------------------------------- decode states --

// A lane holds 16 states of a row (LPR lanes a row of up to 16 LPR states); n states exist.
__device__ __forceinline__ void load_codes16(const int8_t* p, int n, bool vec, float (&f)[16]) {
    if (vec && n >= 16) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = code_at(u[i / 4], i % 4);
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = i < n ? (float)p[i] : 0.f;
}
__device__ __forceinline__ void store_codes16(int8_t* p, int n, bool vec, const int (&q)[16]) {
    if (vec && n >= 16) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]),
                       pack4(q[8], q[9], q[10], q[11]), pack4(q[12], q[13], q[14], q[15]));
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) p[i] = (int8_t)q[i];
}

// 16 values of a row, n of which exist.
template <typename T>
__device__ __forceinline__ void load16(const T* p, int n, float (&f)[16]) {
    load_run<T, 16>(p, 1, 0, n, f);
}

// Codes and scale of a row whose states the LPR lanes hold, written to the cache.
template <int LPR>
__device__ __forceinline__ void put_row(const CacheParams& p, int64_t at, int64_t brow, int j, int n,
                                        bool vec, bool write, const float (&h)[16]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) top = max(top, mag_bits(h[i]));
#pragma unroll
    for (int w = 1; w < LPR; w *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, w));
    if (!write) return;
    const Quant qz(top);
    int q[16];
    if (p.rand) {
        const uint32_t r = p.rand[brow] + (uint32_t)(16 * j) * 0x9E3779B9u;
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = i < n ? qz.dithered(h[i], r + (uint32_t)i * 0x9E3779B9u) : 0;
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = i < n ? qz.nearest(h[i]) : 0;
    }
    store_codes16(p.codes + at * p.dstate + 16 * j, n, vec, q);
    if (j == 0) p.scales[at] = qz.scale;
}

__device__ __forceinline__ int64_t slot_of(const CacheParams& p, int64_t b) {
    const int64_t s = p.slots ? p.slots[b] : b;
    return s >= 0 && s < p.num_slots ? s : -1;
}

template <int LPR, bool VEC>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheParams p) {
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x, brow = idx / LPR;
    const int j = (int)(idx % LPR), n = p.dstate - 16 * j;
    const bool in = brow < p.batch * p.dim;
    const int64_t b = in ? brow / p.dim : 0, slot = in ? slot_of(p, b) : -1;
    float h[16];
    load16(p.state + brow * p.dstate + 16 * j, slot >= 0 ? n : 0, h);
    put_row<LPR>(p, slot * p.dim + (brow - b * p.dim), brow, j, n, VEC, slot >= 0 && n > 0, h);
}

template <typename T, int LPR, bool VEC>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheParams p) {
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x, brow = idx / LPR;
    const int j = (int)(idx % LPR), n = p.dstate - 16 * j;
    if (brow >= p.batch * p.dim || n <= 0) return;
    const int64_t b = brow / p.dim, slot = slot_of(p, b);
    if (slot < 0) return;
    const int64_t at = slot * p.dim + (brow - b * p.dim);
    float h[16];
    load_codes16(p.codes + at * p.dstate + 16 * j, n, VEC, h);
    const float s = p.scales[at];
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] *= s;
    store_run<T, 16>(static_cast<T*>(p.out) + brow * p.dstate + 16 * j, 1, 0, n, h);
}

// One decode step on the cache. LPR lanes share a (batch row, channel); each takes the
// row's conv, delta and gate itself, and its 16 states.
template <typename T, int LPR, bool VEC>
__global__ void __launch_bounds__(256) cached_update_kernel(const CacheParams p) {
    using E = Elem<T>;
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x, brow = idx / LPR;
    const int j = (int)(idx % LPR), n = p.dstate - 16 * j;
    const bool in = brow < p.batch * p.dim;
    const int64_t b = in ? brow / p.dim : 0, slot = in ? slot_of(p, b) : -1;
    const int64_t d = brow - b * p.dim, at = slot * p.dim + d;
    float h[16], y = 0.f, u = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = 0.f;
    T win[4];
    if (slot >= 0) {
        const T newest = static_cast<const T*>(p.x)[brow];
        u = E::to_f(newest);
        if (p.conv_w) {
            const T* cs = static_cast<const T*>(p.conv_state) + at * p.conv_width;
            const float* w = p.conv_w + d * p.conv_width;
            float acc = p.conv_b ? p.conv_b[d] : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < p.conv_width) {
                    win[k] = k + 1 < p.conv_width ? cs[k + 1] : newest;
                    acc = fmaf(w[k], E::to_f(win[k]), acc);
                }
            u = silu(acc);
        }
        const float raw = E::to_f(static_cast<const T*>(p.dt)[brow]) + (p.dt_bias ? p.dt_bias[d] : 0.f);
        const float dl = p.softplus ? (raw > 20.f ? raw : softplus(raw)) : raw;
        if (n > 0) {
            float c[16], Bv[16], Cv[16], a[16];
            load_codes16(p.codes + at * p.dstate + 16 * j, n, VEC, c);
            const float s = p.scales[at], du = dl * u;
            load16(static_cast<const T*>(p.Bt) + b * p.dstate + 16 * j, n, Bv);
            load16(static_cast<const T*>(p.Ct) + b * p.dstate + 16 * j, n, Cv);
            if (p.head_dim) {
                const float e = ex2(dl * p.A[d / p.head_dim] * kLog2e);
#pragma unroll
                for (int i = 0; i < 16; ++i) a[i] = e;
            } else {
                load16(p.A + d * p.dstate + 16 * j, n, a);
#pragma unroll
                for (int i = 0; i < 16; ++i) a[i] = ex2(dl * a[i] * kLog2e);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                h[i] = i < n ? fmaf(a[i], c[i] * s, du * Bv[i]) : 0.f;
                y = fmaf(h[i], Cv[i], y);
            }
        }
    }
    __syncwarp();                                              // a row's lanes have read its window
    if (slot >= 0 && j == 0 && p.conv_w) {
        T* cs = static_cast<T*>(p.conv_state) + at * p.conv_width;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < p.conv_width) cs[k] = win[k];
    }
#pragma unroll
    for (int w = 1; w < LPR; w *= 2) y += __shfl_xor_sync(0xffffffffu, y, w);
    put_row<LPR>(p, at, brow, j, n, VEC, slot >= 0 && n > 0, h);
    if (slot >= 0 && j == 0) {
        if (p.D) y = fmaf(p.D[d], u, y);
        if (p.z) y *= silu(E::to_f(static_cast<const T*>(p.z)[brow]));
        static_cast<T*>(p.out)[brow] = E::from_f(y);
    }
}

}  // namespace ssm
