// Launches of the backward scan kernels of one activation type and layout (one translation
// unit each, so that they compile in parallel).
#pragma once

#include "bwd_launch.h"
#include "scan_bwd_kernel.cuh"

namespace ssm {

template <typename K>
inline cudaError_t launch_with_smem(K k, dim3 grid, int threads, int smem, const BwdParams& p, cudaStream_t st) {
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    k<<<grid, threads, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename T, int S, bool CL, bool Q8, bool HEADS>
inline cudaError_t launch_scan_bwd_v(int what, const BwdParams& p, cudaStream_t st) {
    using H = BwdShape<S>;
    using M = BwdSmem<T, S, CL, Q8, HEADS>;
    constexpr int kRaw = M::kRaw, kHead = M::kHead;
    const dim3 grid((p.dim + H::G - 1) / H::G, p.batch, p.nseg);
    if (what == 0)
        return launch_with_smem(scan_bwd_states_kernel<T, S, CL, Q8, HEADS, kCheckpoint>, grid, H::NT,
                                2 * H::kStaged(false, HEADS) * 4 + kHead + 2 * kRaw +
                                    BwdCopies<T, S, CL, Q8, false>::COUNT * 16,
                                p, st);
    if (what == 1)
        return launch_with_smem(scan_bwd_states_kernel<T, S, CL, Q8, HEADS, kSummary>, grid, H::NT,
                                2 * H::kStaged(true, HEADS) * 4 + kHead + 2 * kRaw +
                                    BwdCopies<T, S, CL, Q8, true>::COUNT * 16,
                                p, st);
    return launch_with_smem(scan_bwd_kernel<T, S, CL, Q8, HEADS>, grid, H::NT, M::kSweep, p, st);
}

template <typename T, bool CL, bool Q8>
inline cudaError_t launch_scan_bwd_t(int what, int lanes, bool heads, const BwdParams& p, cudaStream_t st) {
#define SSM_BWD(S_)                                                                           \
    if (lanes == S_)                                                                          \
        return heads ? launch_scan_bwd_v<T, S_, CL, Q8, true>(what, p, st)                        \
                     : launch_scan_bwd_v<T, S_, CL, Q8, false>(what, p, st);
    SSM_BWD(1) SSM_BWD(2) SSM_BWD(4) SSM_BWD(8) SSM_BWD(16) SSM_BWD(32)
#undef SSM_BWD
    return cudaErrorInvalidValue;
}

}  // namespace ssm
