// Parameters of the 8-bit kernels (activations kept for a backward pass, decode states).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssm {

struct PackParams {
    const void* x;                // pack: the activation; unpack: unused
    int64_t sx;                   // channel-last: elements between positions of x
    int8_t* codes;
    float* scales;
    void* out;                    // unpack
    int batch, dim, seqlen;
    int vec;                      // channel-last x: runs of 8 channels are aligned to their size
};

struct CacheParams {
    int64_t batch, dim, num_slots;
    int dstate;
    int8_t* codes;
    float* scales;
    const int32_t* slots;
    const uint32_t* rand;
    const float* state;           // write
    int vec;                      // write: rows of whole aligned lanes (dstate 8, 16, 32, 64 or 128)
    void* out;                    // read, update
    // update
    void* conv_state;
    const void *x, *dt, *Bt, *Ct, *z;
    const float *A, *D, *dt_bias, *conv_w, *conv_b;
    int conv_width, softplus, head_dim;
    int async;                    // 16-byte aligned codes of 16 states; conv_width 4, aligned, or none
    int rows_per_cta;             // batch rows of a CTA
    int64_t first_row;            // of the launch
};

cudaError_t launch_pack(int elem_size, bool channel_last, const PackParams& p, cudaStream_t st);
cudaError_t launch_unpack(int elem_size, bool channel_last, const PackParams& p, cudaStream_t st);
cudaError_t launch_cache_write(const CacheParams& p, cudaStream_t st);
cudaError_t launch_cache_read(int elem_size, const CacheParams& p, cudaStream_t st);
cudaError_t launch_cached_update(int elem_size, CacheParams p, cudaStream_t st);

}  // namespace ssm
