// 8-bit kernels for sm_100a: activations packed for a backward pass, and the decode states'
// cache. A group (64 positions of a channel, or a channel's row of states) is held as int8
// codes round(127 x / max|x|) and one fp32 scale max|x| / 127. Each value is read once and
// each code written once; what binds is the issue slots (B8 D1536 L2048 bf16: pack 24 us, 83 %
// busy, unpack 17 us, 79 %; HBM alone would take 11.5 each).
//
// Rounding. x (127 / max) + 1.5 2^23 in one fused operation leaves the rounded quotient in
// the sum's low bits. The reciprocal is the SFU's (relative error below 2^-22), so the
// quotient is off by less than 127 2^-22 = 3e-5 and the code is decided unless the quotient
// lies within 5e-5 of a border m = k + 1/2. There the sign of 127 x - m max decides, exactly:
// m max = p + e by a product and its fused remainder, 127 x - p is exact in one fused
// operation (both are near each other), and the two small numbers compare. Ties are common,
// not rare: among bf16 values x = max / 2 alone is met once in some 200.
#pragma once

#include "device_common.cuh"
#include "quant_params.h"
#include "scan_bwd_kernel.cuh"

namespace ssm {

constexpr float kTiny8 = 7.888609052210118e-31f;               // 2^-100

// The largest of |m|, |x|, |y|; NaN if one is.
__device__ __forceinline__ float max_mag(float m, float x, float y) {
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(x), "f"(y));
    return m;
}
template <int N> __device__ __forceinline__ float max_mag(const float (&x)[N]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) m = max_mag(m, x[i], x[i + 1]);
    return m;
}

constexpr float kMagic = 12582912.f;                           // 1.5 2^23
constexpr float kNear = 0.49995f;                              // distance from the rounded quotient

// Codes of a group of values whose largest magnitude is top.
struct Quant {
    float top, inv;
    __device__ __forceinline__ explicit Quant(float largest) : top(largest) {
        // 0 for a group of zeros (in effect: codes 0), or one that is not finite (codes of no
        // matter: the scale is NaN)
        inv = top >= kTiny8 && top < INFINITY ? (127.f / 128.f) * rcp_approx(top * 0.0078125f) : 0.f;
    }
    // top / 127 correctly rounded: the product with 1 / 127 and one correction from its exact
    // remainder (equal to the division for every mantissa)
    __device__ __forceinline__ float scale() const {
        constexpr float c = 1.f / 127.f;
        const float q = top * c, s = fmaf(fmaf(-127.f, q, top), c, q);
        return !(top < INFINITY) ? __uint_as_float(0x7fffffffu) : inv == 0.f ? 0.f : s;
    }
    // round(127 x / top), ties to even; words whose low byte is the code
    template <int N> __device__ __forceinline__ void nearest(const float (&x)[N], uint32_t (&q)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = fmaf(x[i], inv, kMagic);
            const float k = t - kMagic, err = fmaf(x[i], inv, -k);
            q[i] = __float_as_uint(t);
            if (fabsf(err) > kNear) q[i] = (uint32_t)border(x[i], k + copysignf(0.5f, err));
        }
    }
    // The same for values that are hardly ever next to a border (fp32 states): one test for
    // all N, pairs at a time. Without EXACT (a state just computed, which carries roundings of
    // its own) the reciprocal takes a step of Newton's, and the fp32 quotient, off by less than
    // 1e-5 (127 times two roundings of 2^-24 or so), decides borders too.
    template <bool EXACT, int N> __device__ __forceinline__ void nearest_rare(const float (&x)[N], uint32_t (&q)[N]) const {
        const float by = EXACT ? inv : fmaf(inv * (1.f / 127.f), lacking(), inv);
        const uint64_t inv2 = pk2(by, by), magic2 = pk2(kMagic, kMagic), minus = pk2(-1.f, -1.f);
        float worst = 0.f;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint64_t x2 = pk2(x[i], x[i + 1]), t = fma2(x2, inv2, magic2);
            if constexpr (EXACT) {
                const float2 err = upk2(fma2(x2, inv2, fma2(t, minus, magic2)));
                worst = max_mag(worst, err.x, err.y);
            }
            const float2 f = upk2(t);
            q[i] = __float_as_uint(f.x);
            q[i + 1] = __float_as_uint(f.y);
        }
        if (EXACT && worst > kNear) nearest(x, q);             // (NaN: a row that is not finite)
    }
    // floor(127 x / top + offset), the offset of value i the top 24 bits of bits + i GOLDEN as
    // a fraction. F = 1 + offset (to 23 bits: the 24th counts next to a border only) comes out
    // of one funnel shift, and x inv + F plus 1.5 2^23 - 1, rounded down, holds the code.
    // EXACT: offsets are random, so quotients next to a border are rare: fp64 there. Otherwise
    // the quotient gets what the reciprocal lacks, x (inv + lo) + F with the inner sum rounded to
    // the nearest (at most 2^-24, 2^-23 above 2) and the outer one down, which takes no whole
    // number from the sum: the code is the floor of the sum to 3e-7 of a step, and right on
    // average to that. lo is 2^-30 of the reciprocal smaller (1.2e-7 for x = top), more than the
    // inner rounding, so that top itself never comes out as 128 or -128. (Quotients without lo,
    // 2^-21 smaller to stay below 128, lost 5e-7 of every state per step.)
    template <bool EXACT, int N>
    __device__ __forceinline__ void dithered(const float (&x)[N], uint32_t bits, uint32_t (&q)[N]) const {
        const float lo = EXACT ? 0.f : inv * fmaf(lacking(), 1.f / 127.f, -0x1p-30f);
        const uint64_t inv2 = pk2(inv, inv), lo2 = pk2(lo, lo);
        const uint64_t magic2 = pk2(kMagic - 1.f, kMagic - 1.f), minus = pk2(-1.f, -1.f);
        const uint64_t half2 = pk2(-0.5f, -0.5f);
        float worst = 0.f;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint32_t b0 = bits + (uint32_t)i * 0x9E3779B9u, b1 = bits + (uint32_t)(i + 1) * 0x9E3779B9u;
            const uint64_t f2 = pk2(__uint_as_float(__funnelshift_r(b0, 0x7fu, 9)),
                                    __uint_as_float(__funnelshift_r(b1, 0x7fu, 9)));
            const uint64_t x2 = pk2(x[i], x[i + 1]);
            uint64_t v, t;
            if constexpr (EXACT) v = fma2(x2, inv2, f2);
            else asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(x2), "l"(inv2), "l"(fma2(x2, lo2, f2)));
            asm("add.rm.f32x2 %0, %1, %2;" : "=l"(t) : "l"(v), "l"(magic2));
            if constexpr (EXACT) {                             // v less its floor, less a half
                const float2 e = upk2(add2(add2(v, half2), fma2(t, minus, magic2)));
                worst = max_mag(worst, e.x, e.y);
            }
            const float2 f = upk2(t);
            q[i] = __float_as_uint(f.x);
            q[i + 1] = __float_as_uint(f.y);
        }
        if (EXACT && worst > kNear && inv != 0.f) {
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                float v = x[0];
#pragma unroll
                for (int k = 1; k < N; ++k) v = i == k ? x[k] : v;
                const uint32_t b = bits + (uint32_t)i * 0x9E3779B9u;
                const float r = fmaf(v, inv, __uint_as_float(__funnelshift_r(b, 0x7fu, 9)));
                if (fabsf(r - 0.5f - floorf(r)) <= kNear) continue;
                const double o = (double)(b >> 8) * 0x1p-24;
                const uint32_t c = (uint32_t)(int)floor(__ddiv_rn(127.0 * (double)v, (double)top) + o);
#pragma unroll
                for (int k = 0; k < N; ++k) q[k] = i == k ? c : q[k];
            }
        }
    }

  private:
    // 127 - top inv: what the reciprocal lacks (or has too much), times top
    __device__ __forceinline__ float lacking() const { return inv == 0.f ? 0.f : fmaf(-top, inv, 127.f); }
    // the code of x, whose quotient lies next to m = k + 1/2
    __device__ __forceinline__ int border(float x, float m) const {
        const float sc = top > 1.f ? 0.0009765625f : 1.f;      // keeps 127 top finite
        const float xs = x * sc, ts = top * sc, p = m * ts;
        const float e = fmaf(m, ts, -p), d = fmaf(127.f, xs, -p);
        const int lo = (int)(m - 0.5f);
        return d > e ? lo + 1 : d < e ? lo : lo + (lo & 1);
    }
};

// The low bytes of four words.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// Four codes as two pairs of floats: a byte plus 128 in the low bits of 2^23, less 2^23 + 128.
__device__ __forceinline__ void unpack4(uint32_t w, uint64_t (&v)[2]) {
    w ^= 0x80808080u;
    const uint64_t less = pk2(-8388736.f, -8388736.f);
    v[0] = add2(pk2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440)),
                    __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441))), less);
    v[1] = add2(pk2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7442)),
                    __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7443))), less);
}

// N codes of a run (8 or 16): whole and aligned in one access, else byte by byte.
template <int N>
__device__ __forceinline__ void store_codes(int8_t* p, int hi, const uint32_t (&q)[N]) {
    static_assert(N == 8 || N == 16, "one access");
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = pack4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
    if (hi >= N && (reinterpret_cast<uintptr_t>(p) & (N - 1)) == 0) {
        if constexpr (N == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < hi) p[i] = (int8_t)(w[i / 4] >> 8 * (i % 4));
}
// The same codes as words of four; those past hi are 0.
template <int N>
__device__ __forceinline__ void load_code_words(const int8_t* p, int hi, uint32_t (&w)[N / 4]) {
    static_assert(N == 8 || N == 16, "one access");
    if (hi >= N && (reinterpret_cast<uintptr_t>(p) & (N - 1)) == 0) {
        if constexpr (N == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x;
            w[1] = v.y;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (4 * i + k < hi) w[i] |= (uint32_t)(uint8_t)p[4 * i + k] << 8 * k;
    }
}
template <int N>
__device__ __forceinline__ void load_codes(const int8_t* p, int hi, float (&f)[N]) {
    uint32_t w[N / 4];
    load_code_words<N>(p, hi, w);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        uint64_t v[2];
        unpack4(w[i], v);
        f[4 * i] = lo2(v[0]);
        f[4 * i + 1] = hi2(v[0]);
        f[4 * i + 2] = lo2(v[1]);
        f[4 * i + 3] = hi2(v[1]);
    }
}

// ------------------------------------------------------------------ activations --

// i / n and i % n; in 32 bits where i allows it (a 64-bit division takes some 80 instructions).
__device__ __forceinline__ void divide(int64_t i, uint32_t n, int64_t& q, int& r) {
    if (i >> 32 == 0) {
        const uint32_t k = (uint32_t)i / n;
        q = k;
        r = (int)((uint32_t)i - k * n);
    } else {
        q = i / n;
        r = (int)(i - q * n);
    }
}

// (batch, dim, seqlen): 8 neighbouring lanes hold a block of 64 positions.
template <typename T>
__global__ void __launch_bounds__(256) pack_row_kernel(const PackParams p) {
    const int nb = (p.seqlen + kBlock8 - 1) / kBlock8;
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x, blk = idx / 8;
    const int64_t rows = (int64_t)p.batch * p.dim;
    const bool in = blk < rows * nb;
    int64_t row;
    int first;
    divide(in ? blk : 0, nb, row, first);
    const int t = in ? first * kBlock8 + (int)(idx % 8) * 8 : p.seqlen;
    const int hi = min(8, p.seqlen - t);
    float x[8];
    load_run<T, 8>(static_cast<const T*>(p.x) + row * p.seqlen + t, hi, x);
    float top = max_mag(x);
#pragma unroll
    for (int w = 1; w < 8; w *= 2) top = max_mag(top, top, __shfl_xor_sync(0xffffffffu, top, w));
    const Quant qz(top);
    uint32_t q[8];
    qz.nearest(x, q);
    store_codes<8>(p.codes + row * p.seqlen + t, hi, q);
    if (in && idx % 8 == 0) p.scales[blk] = qz.scale();
}

// Channel-last: a warp takes 8 positions of 256 channels (8 a lane), a CTA of 8 warps one
// block of 64 positions; the warps' maxima meet in shared memory.
template <typename T>
__global__ void __launch_bounds__(256) pack_cl_kernel(const PackParams p) {
    __shared__ float tops[8][256];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int d = blockIdx.x * 256 + lane * 8, b = blockIdx.z;
    const int nb = (p.seqlen + kBlock8 - 1) / kBlock8;
    const int hi = min(8, p.dim - d);
    for (int blk = blockIdx.y; blk < nb; blk += gridDim.y) {
        const int t0 = blk * kBlock8 + warp * 8;
        float x[8][8];                                         // [channel][position]
        float top[8];
        const T* src = static_cast<const T*>(p.x) + (int64_t)b * p.seqlen * p.sx + d;
        if (p.vec && hi == 8) {                                // every load before the first use
            float v[8][8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                take_run<T, 8>(src + (int64_t)min(t0 + r, p.seqlen - 1) * p.sx, false, v[r]);
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i][r] = t0 + r < p.seqlen ? v[r][i] : 0.f;
        } else {
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i][r] = t0 + r < p.seqlen && i < hi ? Elem<T>::to_f(src[(int64_t)(t0 + r) * p.sx + i]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) tops[warp][i * 32 + lane] = max_mag(x[i]);
        __syncthreads();
        uint32_t q[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            top[i] = 0.f;
#pragma unroll
            for (int w = 0; w < 8; w += 2)
                top[i] = max_mag(top[i], tops[w][i * 32 + lane], tops[w + 1][i * 32 + lane]);
            const Quant qz(top[i]);
            qz.nearest(x[i], q[i]);
            if (warp == 0 && i < hi) p.scales[((int64_t)b * nb + blk) * p.dim + d + i] = qz.scale();
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = q[i][r];
            if (t0 + r < p.seqlen)
                store_codes<8>(p.codes + ((int64_t)b * p.seqlen + t0 + r) * p.dim + d, hi, v);
        }
    }
}

// A thread reads 8 values back, along the positions of a channel or along the channels.
template <typename T, bool CL>
__global__ void __launch_bounds__(256) unpack_kernel(const PackParams p) {
    const int inner = CL ? p.dim : p.seqlen, runs = (inner + 7) / 8;
    int64_t row;
    int run;
    divide((int64_t)blockIdx.x * 256 + threadIdx.x, runs, row, run);
    const int nb = (p.seqlen + kBlock8 - 1) / kBlock8;
    if (row >= (int64_t)p.batch * (CL ? p.seqlen : p.dim)) return;
    const int k = run * 8, hi = min(8, inner - k);
    float f[8];
    load_codes<8>(p.codes + row * inner + k, hi, f);
    if constexpr (CL) {
        int64_t b;
        int t;
        divide(row, p.seqlen, b, t);
        const int blk = t / kBlock8;
        float s[8];
        load_run<float, 8>(p.scales + (b * nb + blk) * p.dim + k, hi, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= s[i];
    } else {
        const float s = p.scales[row * nb + k / kBlock8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= s;
    }
    store_run<T, 8>(static_cast<T*>(p.out) + row * inner + k, hi, f);
}

// ----------------------------------------------------------------- decode states --

__device__ __forceinline__ int64_t slot_of(const CacheParams& p, int64_t b) {
    const int64_t s = p.slots ? p.slots[b] : b;
    return s >= 0 && s < p.num_slots ? s : -1;
}

// Codes of a row's NP states from first on, and what the row's scale comes from, from LPR
// lanes of a row.
template <bool EXACT, int LPR, int NP>
__device__ __forceinline__ Quant quantise_row(const float (&h)[NP], bool random, uint32_t bits, int first,
                                              uint32_t (&q)[NP]) {
    float top = max_mag(h);
#pragma unroll
    for (int w = 1; w < LPR; w *= 2) top = max_mag(top, top, __shfl_xor_sync(0xffffffffu, top, w));
    const Quant qz(top);
    if (random) qz.dithered<EXACT>(h, bits + (uint32_t)first * 0x9E3779B9u, q);
    else qz.nearest_rare<EXACT>(h, q);
    return qz;
}

// States to codes. A lane takes 8 states of a row, LPR lanes a row (8 LPR states), two rows
// at a time. Row numbers stay below 2^31: 32-bit divisions.
constexpr int kCacheRows = 2;
template <int LPR>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheParams p) {
    constexpr uint32_t per = 256 / LPR;
    const uint32_t rows = (uint32_t)(p.batch * p.dim), dim = (uint32_t)p.dim;
    const int j = threadIdx.x % LPR, n = p.dstate - 8 * j;
    const uint32_t r0 = blockIdx.x * per * kCacheRows + threadIdx.x / LPR;
    float h[kCacheRows][8];
    int64_t at[kCacheRows];                                    // row in the cache, or -1
    uint32_t bits[kCacheRows];
#pragma unroll
    for (int k = 0; k < kCacheRows; ++k) {
        const uint32_t row = r0 + k * per;
        at[k] = -1;
        if (row < rows) {
            const uint32_t b = row / dim;
            const int64_t slot = slot_of(p, b);
            if (slot >= 0) at[k] = slot * dim + (row - b * dim);
        }
    }
    // a padded row's state and rounding bits are not read: they need not exist
#pragma unroll
    for (int k = 0; k < kCacheRows; ++k) {
        const uint32_t row = r0 + k * per;
        const bool live = at[k] >= 0;
        bits[k] = p.rand && live ? p.rand[row] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = 0.f;
        if (p.vec) {
            if (live) take_run<float, 8>(p.state + (int64_t)row * p.dstate + 8 * j, false, h[k]);
        } else {
            load_run<float, 8>(p.state + (int64_t)row * p.dstate + 8 * j, live ? n : 0, h[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < kCacheRows; ++k) {
        uint32_t q[8];
        const Quant qz = quantise_row<true, LPR, 8>(h[k], p.rand != nullptr, bits[k], 8 * j, q);
        if (at[k] < 0) continue;
        if (n > 0) store_codes<8>(p.codes + at[k] * p.dstate + 8 * j, n, q);
        if (j == 0) p.scales[at[k]] = qz.scale();
    }
}

// Codes to states: a thread reads 8 states of a row (LPR threads a row).
template <typename T, int LPR>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheParams p) {
    const uint32_t brow = blockIdx.x * (256 / LPR) + threadIdx.x / LPR, dim = (uint32_t)p.dim;
    const int j = threadIdx.x % LPR, n = p.dstate - 8 * j;
    if (brow >= (uint32_t)(p.batch * p.dim) || n <= 0) return;
    const uint32_t b = brow / dim;
    const int64_t slot = slot_of(p, b);
    if (slot < 0) return;
    const int64_t at = slot * dim + (brow - b * dim);
    float h[8];
    load_codes<8>(p.codes + at * p.dstate + 8 * j, n, h);
    const float s = p.scales[at];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] *= s;
    store_run<T, 8>(static_cast<T*>(p.out) + (int64_t)brow * p.dstate + 8 * j, n, h);
}

// One decode step on the cache. A thread holds 16 states of a channel (LPR threads a
// channel): it keeps the channel's A, conv taps, D and dt bias in registers and takes one
// batch row after the other, the next row's loads issued before the present row is worked
// out. ASYNC: codes, scale, conv window and rounding bits come through a ring of asynchronous
// copies kUpdateStages - 1 rows ahead (rows of 16-byte aligned codes, conv width 4 or none);
// a thread reads back only what it copied itself. The rows' B and C are staged once as fp32
// for all channels of the CTA. B256 D5120 N16 bf16 with conv and rounding bits: 30 us, 94 MB
// (14 us of HBM); the issue slots bind (one row a thread with plain loads: 124 us; without the
// random rounding's second product, biased: 28 us; with
// quotients next to a border decided exactly: 43 us).
constexpr int kUpdateThreads = 128;
constexpr int kUpdateCtas = 4;                                 // per SM: 128 registers a thread
// Most batch rows of a CTA (their B and C take 8 KB at most).
constexpr int update_rows(int lanes) { return lanes >= 8 ? 8 : 64 / lanes < 32 ? 64 / lanes : 32; }
constexpr int kUpdateStages = 4;

template <int N> __device__ __forceinline__ void cp_async_wait_group() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int LPR, bool ASYNC, bool HEADS>
__global__ void __launch_bounds__(kUpdateThreads, kUpdateCtas) cached_update_kernel(const CacheParams p) {
    using E = Elem<T>;
    constexpr int CH = kUpdateThreads / LPR, NS = 16 * LPR;
    __shared__ __align__(16) float bc[update_rows(LPR)][2][NS];
    __shared__ int slot_sm[update_rows(LPR)];
    constexpr int RING = ASYNC ? kUpdateStages : 1;
    __shared__ __align__(16) uint4 ring_codes[RING][ASYNC ? kUpdateThreads : 1];
    __shared__ __align__(16) T ring_conv[RING][ASYNC ? kUpdateThreads : 1][4];
    __shared__ float ring_scale[RING][ASYNC ? kUpdateThreads : 1];
    __shared__ uint32_t ring_rand[RING][ASYNC ? kUpdateThreads : 1];
    const int j = threadIdx.x % LPR, n = p.dstate - 16 * j;
    const int64_t d = (int64_t)blockIdx.x * CH + threadIdx.x / LPR;
    const int64_t b0 = p.first_row + (int64_t)blockIdx.y * p.rows_per_cta;
    const int rows = (int)min((int64_t)p.rows_per_cta, p.batch - b0);
    const bool in = d < p.dim;
    for (int k = threadIdx.x; k < rows * 2 * NS; k += kUpdateThreads) {
        const int r = k / (2 * NS), which = k / NS % 2, i = k % NS;
        const T* src = static_cast<const T*>(which ? p.Ct : p.Bt);
        const bool read = i < p.dstate && slot_of(p, b0 + r) >= 0;  // nothing of a padded row
        bc[r][which][i] = read ? E::to_f(src[(b0 + r) * p.dstate + i]) : 0.f;
    }
    if (threadIdx.x < rows) slot_sm[threadIdx.x] = (int)slot_of(p, b0 + threadIdx.x);
    float A2[16], w[4], cb = 0.f, Dv = 0.f, bias = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int kk = k - (4 - p.conv_width);                 // right-aligned taps
        w[k] = in && kk >= 0 ? p.conv_w[d * p.conv_width + kk] : 0.f;
    }
    if (in) {
        if (p.conv_b) cb = p.conv_b[d];
        if (p.D) Dv = p.D[d];
        if (p.dt_bias) bias = p.dt_bias[d];
        if constexpr (HEADS) {
            const float a = p.A[d / p.head_dim] * kLog2e;
#pragma unroll
            for (int i = 0; i < 16; ++i) A2[i] = a;
        } else {
            load_run<float, 16>(p.A + d * p.dstate + 16 * j, n, A2);
#pragma unroll
            for (int i = 0; i < 16; ++i) A2[i] *= kLog2e;
        }
    }
    __syncthreads();

    struct Row {                                               // one row's inputs, as they come
        uint32_t codes[4], rand;
        float scale, win[3];                                   // win: the last 3 conv inputs
        T x, dt, z;
        int slot;
    };
    // rows of the cache and of the batch count below 2^32: one wide multiply-add an address
    const uint32_t dim = (uint32_t)p.dim, ch = (uint32_t)d, row0 = (uint32_t)b0 * dim + ch;
    auto codes_at = [&](uint32_t at) { return p.codes + 16 * j + (uint64_t)at * (uint32_t)p.dstate; };
    auto conv_at = [&](uint32_t at) { return static_cast<T*>(p.conv_state) + (uint64_t)at * (uint32_t)p.conv_width; };
    auto load = [&](int r, Row& v) {
        v.slot = -1;
        if (r >= rows || !in) return;
        v.slot = slot_sm[r];
        if (v.slot < 0) return;
        const uint32_t brow = row0 + r * dim, at = v.slot * dim + ch;
        v.x = static_cast<const T*>(p.x)[brow];
        v.dt = static_cast<const T*>(p.dt)[brow];
        if (p.z) v.z = static_cast<const T*>(p.z)[brow];
        if constexpr (!ASYNC) {
            load_code_words<16>(codes_at(at), n, v.codes);
            v.scale = p.scales[at];
            if (p.rand) v.rand = p.rand[brow];
            if (p.conv_w) {
                const T* cs = conv_at(at);
#pragma unroll
                for (int k = 0; k < 3; ++k) {                  // input at lag 3 - k
                    const int kk = p.conv_width - 3 + k;
                    v.win[k] = kk >= 1 ? E::to_f(cs[kk]) : 0.f;
                }
            }
        }
    };
    auto copy = [&](int r) {                                   // ASYNC: row r into its ring place
        const int slot = r < rows && in ? slot_sm[r < rows ? r : 0] : -1;
        if (slot >= 0) {
            const int st = r % RING, tid = ASYNC ? threadIdx.x : 0;
            const uint32_t at = slot * dim + ch;
            cp_async<16>(smem_u32(&ring_codes[st][tid]), n > 0 ? codes_at(at) : p.codes, n > 0 ? 16 : 0);
            cp_async<4>(smem_u32(&ring_scale[st][tid]), p.scales + at, 4);
            if (p.conv_w)
                cp_async<4 * (int)sizeof(T)>(smem_u32(&ring_conv[st][tid]), conv_at(at), 4 * (int)sizeof(T));
            if (p.rand) cp_async<4>(smem_u32(&ring_rand[st][tid]), p.rand + (row0 + r * dim), 4);
        }
        cp_async_commit();
    };
    if constexpr (ASYNC) {
#pragma unroll
        for (int r = 0; r < kUpdateStages - 1; ++r) copy(r);
    }
    Row next, after;                                           // two rows ahead
    load(0, next);
    load(1, after);
    for (int r = 0; r < rows; ++r) {
        Row v = next;
        next = after;
        load(r + 2, after);
        const bool live = v.slot >= 0;
        const uint32_t at = v.slot * dim + ch;
        if constexpr (ASYNC) {
            copy(r + kUpdateStages - 1);
            cp_async_wait_group<kUpdateStages - 1>();
            if (live) {
                const int st = r % RING, tid = threadIdx.x;
                const uint4 c = ring_codes[st][tid];
                v.codes[0] = c.x;
                v.codes[1] = c.y;
                v.codes[2] = c.z;
                v.codes[3] = c.w;
                v.scale = ring_scale[st][tid];
                if (p.rand) v.rand = ring_rand[st][tid];
                if (p.conv_w) {
                    float f[4];
                    take_run<T, 4>(ring_conv[st][tid], false, f);
#pragma unroll
                    for (int k = 0; k < 3; ++k) v.win[k] = f[k + 1];
                }
            }
        }
        __syncwarp();                                          // a row's lanes hold its window
        float h[16], y = 0.f, u = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = 0.f;
        if (live) {
            u = E::to_f(v.x);
            if (p.conv_w) {
                float acc = fmaf(w[3], u, cb);
#pragma unroll
                for (int k = 0; k < 3; ++k) acc = fmaf(w[k], v.win[k], acc);
                if (j == 0) {
                    T* cs = conv_at(at);
                    const float win[4] = {v.win[0], v.win[1], v.win[2], u};
                    if constexpr (ASYNC) {
                        put_run<T, 4>(cs, false, true, 4, win);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k >= 4 - p.conv_width) cs[k - (4 - p.conv_width)] = E::from_f(win[k]);
                    }
                }
                u = silu(acc);
            }
            const float raw = E::to_f(v.dt) + bias;
            const float dl = p.softplus ? (raw > 20.f ? raw : softplus(raw)) : raw;
            const uint64_t d2 = pk2(dl, dl), du2 = pk2(dl * u, dl * u), s2 = pk2(v.scale, v.scale);
            const ulonglong2* Bv = reinterpret_cast<const ulonglong2*>(bc[r][0] + 16 * j);
            const ulonglong2* Cv = reinterpret_cast<const ulonglong2*>(bc[r][1] + 16 * j);
            uint64_t y2 = 0;
            float one = 0.f;                                   // A per head: one decay
            if constexpr (HEADS) one = ex2(dl * A2[0]);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint64_t c[2];
                unpack4(v.codes[g], c);
                const ulonglong2 b2 = Bv[g], c2 = Cv[g];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = 4 * g + 2 * k;
                    uint64_t a = pk2(one, one);
                    if constexpr (!HEADS) {
                        const float2 e = upk2(mul2(d2, pk2(A2[i], A2[i + 1])));
                        a = pk2(ex2(e.x), ex2(e.y));
                    }
                    const uint64_t hn = fma2(a, mul2(c[k], s2), mul2(du2, k ? b2.y : b2.x));
                    y2 = fma2(hn, k ? c2.y : c2.x, y2);
                    const float2 f = upk2(hn);
                    h[i] = f.x;
                    h[i + 1] = f.y;
                }
            }
            const float2 f = upk2(y2);
            y = f.x + f.y;
        }
#pragma unroll
        for (int k = 1; k < LPR; k *= 2) y += __shfl_xor_sync(0xffffffffu, y, k);
        uint32_t q[16];
        const Quant qz = quantise_row<false, LPR, 16>(h, p.rand != nullptr, v.rand, 16 * j, q);
        if (!live) continue;
        if (n > 0) store_codes<16>(codes_at(at), n, q);
        if (j == 0) {
            p.scales[at] = qz.scale();
            y = fmaf(Dv, u, y);
            if (p.z) y *= silu(E::to_f(v.z));
            static_cast<T*>(p.out)[row0 + r * dim] = E::from_f(y);
        }
    }
}

}  // namespace ssm
