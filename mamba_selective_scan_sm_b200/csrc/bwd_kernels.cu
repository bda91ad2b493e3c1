// The backward pass's small kernels (carry chain, reductions, sequence starts) and the
// conv's gradient.
#define SSM_ERROR_WORD g_error_bwd
#include "conv_bwd_kernel.cuh"

#include "bwd_launch.h"

namespace ssm {

// min(position - start of its sequence, 4) for every position of a packed row, from the
// offsets (a binary search per position; offsets out of order or range give some value in
// 0..4, never an access outside).
__global__ void __launch_bounds__(256) since_kernel(const int32_t* cu, int nseq, int seqlen, uint8_t* out) {
    const int t = blockIdx.x * blockDim.x + threadIdx.x;
    if (t >= seqlen) return;
    int lo = 0, hi = nseq;                                     // last s in [0, nseq) with cu[s] <= t
    while (hi - lo > 1) {
        const int m = lo + (hi - lo) / 2;
        if (cu[m] <= t) lo = m;
        else hi = m;
    }
    const int64_t d = (int64_t)t - cu[lo];
    out[t] = (uint8_t)(d < 0 ? 0 : d > 4 ? 4 : d);
}

// dB and dC: the sum over the channel groups of their partial rows, rounded once. A CTA
// takes kReduceSteps steps of one batch row; the sums pass through shared memory, since
// (batch, dstate, seqlen) outputs run along the steps and the partial rows along the states.
constexpr int kReduceSteps = 8;
constexpr int kReduceGroups = 64;  // whose sum is taken by itself: 2^20 channels make 32768 groups
template <typename T>
__global__ void __launch_bounds__(128) scan_bwd_reduce_bc_kernel(const BwdReduceParams p) {
    extern __shared__ float sm[];
    const int row = 2 * p.ns, b = blockIdx.y, t0 = blockIdx.x * kReduceSteps;
    const int nt = min(kReduceSteps, p.seqlen - t0);
    const int64_t gstride = (int64_t)p.batch * p.seqlen * row;
    const float* src = p.parts + ((int64_t)b * p.seqlen + t0) * row;
    for (int k = threadIdx.x * 4; k < nt * row; k += blockDim.x * 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int g0 = 0; g0 < p.groups; g0 += kReduceGroups) {  // in two steps: short chains
            float4 part = make_float4(0.f, 0.f, 0.f, 0.f);
            const int g1 = min(p.groups, g0 + kReduceGroups);
#pragma unroll 8
            for (int g = g0; g < g1; ++g) {
                const float4 q = *reinterpret_cast<const float4*>(src + g * gstride + k);
                part.x += q.x;
                part.y += q.y;
                part.z += q.z;
                part.w += q.w;
            }
            v.x += part.x;
            v.y += part.y;
            v.z += part.z;
            v.w += part.w;
        }
        float* o = sm + (k / row) * (row + 1) + k % row;
        o[0] = v.x;
        o[1] = v.y;
        o[2] = v.z;
        o[3] = v.w;
    }
    __syncthreads();
    const bool along_p = p.sdB.p == 1 && p.sdB.c != 1;
    for (int k = threadIdx.x; k < nt * p.dstate * 2; k += blockDim.x) {
        const int which = k / (nt * p.dstate), r = k % (nt * p.dstate);
        const int n = along_p ? r / nt : r % p.dstate, tl = along_p ? r % nt : r / p.dstate;
        const int pos = p.reverse ? p.seqlen - 1 - (t0 + tl) : t0 + tl;
        const Str& s = which ? p.sdC : p.sdB;
        T* o = static_cast<T*>(which ? p.dC : p.dB);
        o[(int64_t)b * s.b + (int64_t)n * s.c + (int64_t)pos * s.p] =
            Elem<T>::from_f(sm[tl * (row + 1) + which * p.ns + n]);
    }
}

// dA, dD and d delta_bias: sums over the batch rows and segments. A per state: a thread
// per (channel, state) and per channel. A per head: a CTA per head sums over its channels
// and states too.
__global__ void __launch_bounds__(256) scan_bwd_reduce_a_kernel(const BwdReduceParams p) {
    const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t na = p.head_dim ? 0 : (int64_t)p.dim * p.ns;
    if (idx < na) {
        const int d = (int)(idx / p.ns), n = (int)(idx % p.ns) ^ (d >> p.order_shift & p.order_mask);
        if (n >= p.dstate) return;
        LongSum v;
#pragma unroll 8
        for (int r = 0; r < p.nrows; ++r) v.add(p.pA[r * na + idx]);
        p.dA[(int64_t)d * p.dstate + n] = v.get();
    } else if (idx < na + 2 * (int64_t)p.dim) {
        const int64_t k = idx - na;
        float* o = k % 2 ? p.dbias : p.dD;
        if (!o) return;
        LongSum v;
#pragma unroll 8
        for (int r = 0; r < p.nrows; ++r) v.add(p.pD[(int64_t)r * p.dim * 2 + k]);
        o[k / 2] = v.get();
    }
}

__global__ void __launch_bounds__(256) scan_bwd_reduce_heads_kernel(const BwdReduceParams p) {
    const int h = blockIdx.x;
    LongSum sum;
    for (int r = 0; r < p.nrows; ++r) {                        // (nrows, dim): summed over the states
        const float* src = p.pA + (int64_t)r * p.dim + (int64_t)h * p.head_dim;
        for (int k = threadIdx.x; k < p.head_dim; k += blockDim.x) sum.add(src[k]);
    }
    float v = sum.get();
    __shared__ float red[256 / 32];
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = 0.f;
        for (int k = 0; k < 256 / 32; ++k) v += red[k];
        p.dA[h] = v;
    }
}

template <int S, typename T, bool HEADS> static constexpr int ctas_of() {
    constexpr int n = BwdSmem<T, S, false, false, HEADS>::CTAS;
    static_assert(n == BwdSmem<T, S, true, false, HEADS>::CTAS && n == BwdSmem<T, S, false, true, HEADS>::CTAS &&
                      n == BwdSmem<T, S, true, true, HEADS>::CTAS,
                  "the workspace's size goes by neither the layout nor 8-bit inputs");
    return n;
}
template <int S> static BwdVariant variant_of(int elem_size, bool heads) {
    using H = BwdShape<S>;
    using B = __nv_bfloat16;
    const int ctas = elem_size == 2 ? (heads ? ctas_of<S, B, true>() : ctas_of<S, B, false>())
                                    : (heads ? ctas_of<S, float, true>() : ctas_of<S, float, false>());
    return {H::NS, H::G, H::TT, H::T, H::DRAIN, ctas, H::KL - 1, H::NC - 1};
}
BwdVariant scan_bwd_variant(int lanes, int elem_size, bool heads) {
    return lanes == 1   ? variant_of<1>(elem_size, heads)
           : lanes == 2 ? variant_of<2>(elem_size, heads)
           : lanes == 4 ? variant_of<4>(elem_size, heads)
           : lanes == 8 ? variant_of<8>(elem_size, heads)
           : lanes == 16 ? variant_of<16>(elem_size, heads)
                         : variant_of<32>(elem_size, heads);
}

cudaError_t launch_scan_bwd_carry(int ns, const BwdParams& p, cudaStream_t st) {
    const int64_t n = (int64_t)p.batch * p.dim * ns;
    const unsigned blocks = (unsigned)((n + 255) / 256);
#define SSM_BWD(S_)                                                                           \
    if (ns == 4 * S_) {                                                                       \
        scan_bwd_carry_kernel<S_><<<blocks, 256, 0, st>>>(p);                                \
        return cudaGetLastError();                                                            \
    }
    SSM_BWD(1) SSM_BWD(2) SSM_BWD(4) SSM_BWD(8) SSM_BWD(16) SSM_BWD(32)
#undef SSM_BWD
    return cudaErrorInvalidValue;
}

cudaError_t launch_scan_bwd_reduce(int elem_size, const BwdReduceParams& p, cudaStream_t st) {
    const dim3 g((p.seqlen + kReduceSteps - 1) / kReduceSteps, p.batch);
    const int smem = kReduceSteps * (2 * p.ns + 1) * (int)sizeof(float);
    if (elem_size == 2) scan_bwd_reduce_bc_kernel<__nv_bfloat16><<<g, 128, smem, st>>>(p);
    else scan_bwd_reduce_bc_kernel<float><<<g, 128, smem, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t n = (p.head_dim ? 0 : (int64_t)p.dim * p.ns) + 2 * (int64_t)p.dim;
    scan_bwd_reduce_a_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.head_dim) return e;
    scan_bwd_reduce_heads_kernel<<<p.dim / p.head_dim, 256, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_since(const int32_t* cu, int nseq, int seqlen, uint8_t* since, cudaStream_t st) {
    since_kernel<<<(seqlen + 255) / 256, 256, 0, st>>>(cu, nseq, seqlen, since);
    return cudaGetLastError();
}

int conv_bwd_chunk(bool channel_last) { return channel_last ? kConvClChunk : kConvRowChunk; }

cudaError_t launch_conv_bwd(int elem_size, bool channel_last, const ConvBwdParams& p, cudaStream_t st) {
    if (channel_last) {
        const int per = 128 * kConvClRun;
        const dim3 g((unsigned)((p.dim + per - 1) / per) * (unsigned)p.chunks, p.batch);
        const bool q8 = p.x.scale != nullptr;
        if (elem_size == 2) {
            if (q8) conv_bwd_cl_kernel<__nv_bfloat16, true><<<g, 128, 0, st>>>(p);
            else conv_bwd_cl_kernel<__nv_bfloat16, false><<<g, 128, 0, st>>>(p);
        } else {
            if (q8) conv_bwd_cl_kernel<float, true><<<g, 128, 0, st>>>(p);
            else conv_bwd_cl_kernel<float, false><<<g, 128, 0, st>>>(p);
        }
    } else {
        const int64_t rows = (int64_t)p.batch * p.dim;
        const dim3 g(p.chunks, (unsigned)(rows < 65535 ? rows : 65535), (unsigned)((rows + 65534) / 65535));
        const bool q8 = p.x.scale != nullptr;
        if (elem_size == 2) {
            if (q8) conv_bwd_row_kernel<__nv_bfloat16, true><<<g, kConvRowThreads, 0, st>>>(p);
            else conv_bwd_row_kernel<__nv_bfloat16, false><<<g, kConvRowThreads, 0, st>>>(p);
        } else {
            if (q8) conv_bwd_row_kernel<float, true><<<g, kConvRowThreads, 0, st>>>(p);
            else conv_bwd_row_kernel<float, false><<<g, kConvRowThreads, 0, st>>>(p);
        }
    }
    return cudaGetLastError();
}

cudaError_t launch_conv_reduce(const ConvReduceParams& p, cudaStream_t st) {
    conv_reduce_kernel<<<(unsigned)(((int64_t)p.dim * 5 + 31) / 32), 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace ssm
