// Host-side launchers of the backward-pass and 8-bit kernels.
#pragma once

#include <cuda_runtime.h>

#include "bwd_params.h"

namespace ssm {

// Static shape of the backward scan kernels for `lanes` (1, 2, .. 32) lanes per channel.
struct BwdVariant {
    int ns, channels, tile;
    int order_mask;               // scratch states of channel d stand at n ^ (d & order_mask)
};
BwdVariant scan_bwd_variant(int lanes);

// what: 0 checkpoints, 1 segment summaries, 2 the backward sweep.
cudaError_t launch_scan_bwd_bf16(int what, int lanes, bool heads, const BwdParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_f32(int what, int lanes, bool heads, const BwdParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_bf16_cl(int what, int lanes, bool heads, const BwdParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_f32_cl(int what, int lanes, bool heads, const BwdParams& p, cudaStream_t st);

cudaError_t launch_scan_bwd_carry(int ns, const BwdParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_reduce(int elem_size, const BwdReduceParams& p, cudaStream_t st);
cudaError_t launch_since(const int32_t* cu, int nseq, int seqlen, uint8_t* since, cudaStream_t st);

// Positions of a row (or, channel-last, steps) that one CTA of the conv's gradient takes.
int conv_bwd_chunk(bool channel_last);
cudaError_t launch_conv_bwd(int elem_size, bool channel_last, const ConvBwdParams& p, cudaStream_t st);
cudaError_t launch_conv_reduce(const ConvReduceParams& p, cudaStream_t st);

}  // namespace ssm
