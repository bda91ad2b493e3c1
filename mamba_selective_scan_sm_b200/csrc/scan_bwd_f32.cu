// Instantiations of the backward scan kernels: f32 activations, (batch, dim, seqlen) layout, plain u, delta, z.
#define SSM_ERROR_WORD g_error_scan_bwd_f32
#include "scan_bwd_launch.cuh"

namespace ssm {

cudaError_t launch_scan_bwd_f32(int what, int lanes, bool heads, const BwdParams& p, cudaStream_t st) {
    return launch_scan_bwd_t<float, false, false>(what, lanes, heads, p, st);
}

}  // namespace ssm
