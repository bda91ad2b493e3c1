// Host-side launchers of the backward-pass and 8-bit kernels.
#pragma once

#include <cuda_runtime.h>

#include "bwd_params.h"

namespace ssm {

// Static shape of the backward scan kernels for `lanes` (1, 2, .. 32) lanes per channel; ctas
// also goes by the activations' size and A per head (not by the layout or 8-bit inputs).
struct BwdVariant {
    int ns, channels, tile;
    int steps;                    // between two checkpoints of the state
    int drain;                    // tiles between two additions to the sums over a segment
    int ctas;                     // of the backward sweep per SM
    int order_shift, order_mask;  // scratch states of channel d stand at n ^ (d >> shift & mask)
};
BwdVariant scan_bwd_variant(int lanes, int elem_size, bool heads);

// what: 0 checkpoints, 1 segment summaries, 2 the backward sweep. One per activation type,
// layout (_cl: channel-last) and form of u, delta and z (_q8: int8 codes).
#define SSM_DECLARE_BWD(NAME_) \
    cudaError_t launch_scan_bwd_##NAME_(int what, int lanes, bool heads, const BwdParams& p, cudaStream_t st);
SSM_DECLARE_BWD(bf16) SSM_DECLARE_BWD(f32) SSM_DECLARE_BWD(bf16_cl) SSM_DECLARE_BWD(f32_cl)
SSM_DECLARE_BWD(bf16_q8) SSM_DECLARE_BWD(f32_q8) SSM_DECLARE_BWD(bf16_cl_q8) SSM_DECLARE_BWD(f32_cl_q8)
#undef SSM_DECLARE_BWD

cudaError_t launch_scan_bwd_carry(int ns, const BwdParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_reduce(int elem_size, const BwdReduceParams& p, cudaStream_t st);
cudaError_t launch_since(const int32_t* cu, int nseq, int seqlen, uint8_t* since, cudaStream_t st);

// Positions of a row (or, channel-last, steps) that one CTA of the conv's gradient takes.
int conv_bwd_chunk(bool channel_last);
cudaError_t launch_conv_bwd(int elem_size, bool channel_last, const ConvBwdParams& p, cudaStream_t st);
cudaError_t launch_conv_reduce(const ConvReduceParams& p, cudaStream_t st);

}  // namespace ssm
