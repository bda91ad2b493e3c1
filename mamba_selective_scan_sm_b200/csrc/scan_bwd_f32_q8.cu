// Instantiations of the backward scan kernels: f32 activations, (batch, dim, seqlen) layout, int8 u, delta, z.
#define SSM_ERROR_WORD g_error_scan_bwd_f32_q8
#include "scan_bwd_launch.cuh"

namespace ssm {

cudaError_t launch_scan_bwd_f32_q8(int what, int lanes, bool heads, const BwdParams& p, cudaStream_t st) {
    return launch_scan_bwd_t<float, false, true>(what, lanes, heads, p, st);
}

}  // namespace ssm
