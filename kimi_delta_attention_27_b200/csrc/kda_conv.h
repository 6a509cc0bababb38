// Internal interface of the short causal convolution kernels (see include/kda.h, kda_conv_*).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_seq.cuh"

namespace kda {

constexpr int kConvMinTaps = 2, kConvMaxTaps = 4;

struct ConvParams {
    Seqs seqs;
    int64_t rows;            // tokens in all
    int32_t C, W;            // channels (a multiple of 8), taps
    int32_t fp32;            // x, out, states and their gradients: 1 fp32, 0 bf16
    int32_t silu;
    const float *weight;     // [C, W]
    const float *bias;       // [C] or nullptr
    const void *x;           // row r at x + r * x_stride elements
    int64_t x_stride;
    const void *init;        // [n, W - 1, C] or nullptr
    // forward
    void *out;
    int64_t out_stride;
    void *final_state;       // [n, W - 1, C] or nullptr
    // backward
    const void *dout;
    int64_t dout_stride;
    int32_t dout_fp32;
    const void *dfinal;      // [n, W - 1, C] or nullptr
    void *dx;
    int64_t dx_stride;
    void *dinit;             // [n, W - 1, C] or nullptr
    float *dweight, *dbias;  // [C, W], [C] or nullptr
    float *partial;          // [conv_bwd_blocks, W + 1, C]
};

struct ConvDecodeParams {
    int64_t batch;
    int32_t C, W, fp32, silu;
    const float *weight, *bias;
    const void *x;
    int64_t x_stride;
    const void *state_in;    // [batch, W - 1, C] or nullptr (zeros)
    void *state_out;         // [batch, W - 1, C] or nullptr
    void *out;               // [batch, C]
    int64_t out_stride;
};

// token blocks of the backward launch: rows of its partial sums
int32_t conv_bwd_blocks(int64_t rows, int32_t C);
cudaError_t launch_conv_fwd(const ConvParams &p, cudaStream_t stream);
cudaError_t launch_conv_bwd(const ConvParams &p, cudaStream_t stream);
cudaError_t launch_conv_decode(const ConvDecodeParams &p, cudaStream_t stream);
cudaError_t read_and_clear_conv_error(unsigned int *value);

}  // namespace kda
