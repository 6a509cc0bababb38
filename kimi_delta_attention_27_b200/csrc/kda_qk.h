// Internal interface of the q/k norm and rotation kernels (see include/kda.h, kda_qk_*).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kNormNone = 0, kNormL2 = 1, kNormRms = 2;

struct QkParams {
    int64_t rows;                 // tokens
    int32_t Hq, Hk, D;            // D 64, 128 or 256
    int32_t norm;
    float eps;
    const float *q_weight, *k_weight;   // [D] or nullptr
    const int32_t *positions;     // [rows]
    const float *inv_freq;        // [rot / 2]
    int32_t rot;                  // rotated channels, a multiple of 16 (0: none)
    int32_t interleaved;
    float factor;                 // on cos and sin
    const uint16_t *q, *k;        // bf16, row r at q + r * q_stride
    int64_t q_stride, k_stride;
    uint16_t *q_out, *k_out;      // forward: the results; backward: dq, dk
    int64_t q_out_stride, k_out_stride;
    // backward
    const void *dq_out, *dk_out;  // bf16 or fp32
    int64_t dq_stride, dk_stride;
    int32_t dout_fp32;
    float *dq_weight, *dk_weight; // [D] or nullptr
    float *partial;               // [qk_bwd_blocks, 2, D]
};

int32_t qk_bwd_blocks(int64_t rows, int32_t heads, int32_t D);
cudaError_t launch_qk_fwd(const QkParams &p, cudaStream_t stream);
cudaError_t launch_qk_bwd(const QkParams &p, cudaStream_t stream);

}  // namespace kda
