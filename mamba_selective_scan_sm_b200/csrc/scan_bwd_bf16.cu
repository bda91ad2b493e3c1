// Instantiations of the backward scan kernels: bf16 activations, (batch, dim, seqlen) layout, plain u, delta, z.
#define SSM_ERROR_WORD g_error_scan_bwd_bf16
#include "scan_bwd_launch.cuh"

namespace ssm {

cudaError_t launch_scan_bwd_bf16(int what, int lanes, bool heads, const BwdParams& p, cudaStream_t st) {
    return launch_scan_bwd_t<__nv_bfloat16, false, false>(what, lanes, heads, p, st);
}

}  // namespace ssm
