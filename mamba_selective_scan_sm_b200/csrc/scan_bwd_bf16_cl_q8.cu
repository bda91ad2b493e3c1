// Instantiations of the backward scan kernels: bf16 activations, channel-last layout, int8 u, delta, z.
#define SSM_ERROR_WORD g_error_scan_bwd_bf16_cl_q8
#include "scan_bwd_launch.cuh"

namespace ssm {

cudaError_t launch_scan_bwd_bf16_cl_q8(int what, int lanes, bool heads, const BwdParams& p, cudaStream_t st) {
    return launch_scan_bwd_t<__nv_bfloat16, true, true>(what, lanes, heads, p, st);
}

}  // namespace ssm
