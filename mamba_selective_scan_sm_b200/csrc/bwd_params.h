// Parameters of the backward-pass kernels (plain data, shared by host and device code).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssm {

// Element strides of an activation: batch row, channel (or state), position.
struct Str {
    int64_t b, c, p;
};

// An activation the backward pass reads: values in the activation type, or (scale set)
// int8 codes with one fp32 scale per channel and kBlock8 positions.
struct ActIn {
    const void* p;
    const float* scale;
    Str s;        // of the values or codes
    Str ss;       // of the scales; ss.p is the stride between blocks
};

constexpr int kBlock8 = 64;       // positions per scale of an 8-bit activation

struct BwdParams {
    int batch, dim, seqlen, dstate;
    ActIn x, dt, z;               // x: the scan's input u, or the conv's input with conv_w
    const void *dy, *Bm, *Cm;
    Str sdy, sB, sC;
    const float* A;               // (dim, dstate), or (dim / head_dim)
    const float *D, *dbias, *conv_w, *conv_b;
    int conv_width, softplus, reverse, head_dim;
    int async;                    // every row is aligned to the asynchronous copies' unit
    int vec_out;                  // the outputs' runs are aligned to 16 bytes
    const float* h0;              // (batch, dim, dstate) or null
    const float* dhl;             // (batch, dim, dstate) or null: gradient of the last state
    const void* hist;             // (batch, dim, conv_width - 1) or null
    const uint8_t* since;         // (seqlen) or null: min(position - sequence start, 4)
    void* du;                     // gradient of u; with conv_w the fp32 scratch du32 instead
    float* du32;                  // dense, laid out as the activations (channel_last or not)
    void *ddt, *dz;
    Str sdu, sddt, sdz;
    float* dh0;                   // (batch, dim, dstate) or null
    float* ckpt;                  // states before every BwdShape::T-th step
    int nsub;                     // checkpoints per row, of whole tiles
    float* parts;                 // (groups, batch, seqlen, 2, NS): dB, dC of a channel group
    float* pA;                    // (nseg * batch, dim, NS); with A per head (nseg * batch, dim)
    float* pA_lo;                 // as pA, for segments longer than a drain: what its sums round off
    float* pD;                    // (nseg * batch, dim, 2): dD, d delta_bias
    float *sumP, *sumS, *sumR;    // (nseg, batch, dim, NS) segment summaries, then carries
    int nseg, seg_len;
};

// The conv's gradient. dpre = dout * act'(pre); dx_s = sum_k w_k dpre_{s+W-1-k}.
struct ConvBwdParams {
    int batch, dim, seqlen, width;
    ActIn x;
    const void* dout;             // activation type, or fp32 (dout32)
    int dout32;
    Str sdo;
    const float *w, *bias;
    int silu, reverse;
    int vec;                      // runs of x, dout and dx are aligned to their size, rows whole runs
    const void* hist;
    const uint8_t* since;
    void* dx;
    Str sdx;
    void* dhist;                  // (batch, dim, width - 1) or null
    float* part;                  // (batch * chunks, dim, 5): dw (right-aligned), dbias
    int chunks, chunk_len;
};

// Sums the partial results of a backward pass.
struct BwdReduceParams {
    int batch, dim, seqlen, dstate, ns, groups, nrows, reverse, head_dim, order_shift, order_mask;
    const float *parts, *pA, *pD;
    void *dB, *dC;                // in the activations' type
    Str sdB, sdC;
    float *dA, *dD, *dbias;
};

struct ConvReduceParams {
    int dim, width;
    int64_t rows;
    const float* part;
    float *dw, *dbias;
};

}  // namespace ssm
