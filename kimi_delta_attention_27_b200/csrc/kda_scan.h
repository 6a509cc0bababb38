// Internal interface of the selective state space scan kernels (see include/kda.h, kda_scan_*).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_seq.cuh"

namespace kda {

struct ScanParams {
    Seqs seqs;
    int64_t rows;                 // tokens in all
    int32_t H, G, P, N;           // heads, groups of B and C, head channels (64 or 128), state size (64 or 128)
    const uint16_t *x;            // bf16, row r, head h at x + r * x_stride + h * P
    int64_t x_stride;
    const float *dt;              // [rows, H]
    const float *A;               // [H]
    const uint16_t *B, *C;        // bf16, row r, group g at B + r * b_stride + g * N
    int64_t b_stride, c_stride;
    const float *D, *dt_bias;     // [H] or nullptr
    int32_t softplus;
    const void *h0;               // [n, H, N, P] or nullptr
    int32_t h0_fp32;
    void *hT;                     // [n, H, N, P] or nullptr
    int32_t hT_fp32;
    uint16_t *out;                // bf16, row r, head h at out + r * out_stride + h * P
    int64_t out_stride;
    float *ws;                    // scan_fwd_workspace_bytes
    // backward
    const uint16_t *dout;         // bf16, row r, head h at dout + r * dout_stride + h * P
    int64_t dout_stride;
    const float *dhT;             // [n, H, N, P] or nullptr
    uint16_t *dx, *dB, *dC;       // bf16, strided as x, B, C are
    int64_t dx_stride, db_stride, dc_stride;
    float *ddt;                   // [rows, H]
    float *dA, *dD, *ddt_bias;    // [H] (dD, ddt_bias or nullptr)
    float *dh0;                   // [n, H, N, P] or nullptr
};

struct ScanDecodeParams {
    int64_t batch;
    int32_t H, G, P, N;
    const uint16_t *x, *B, *C;
    int64_t x_stride, b_stride, c_stride;
    const float *dt, *A, *D, *dt_bias;
    int32_t softplus;
    const void *state_in;         // [batch, H, N, P] or nullptr (zeros)
    void *state_out;              // or nullptr
    int32_t state_fp32;
    uint16_t *out;                // [batch, H, P]
};

size_t scan_fwd_workspace_bytes(int64_t rows, int64_t n, int32_t H, int32_t P, int32_t N);
size_t scan_bwd_workspace_bytes(int64_t rows, int64_t n, int32_t H, int32_t G, int32_t P, int32_t N);
cudaError_t launch_scan_fwd(const ScanParams &p, cudaStream_t stream);
cudaError_t launch_scan_bwd(const ScanParams &p, cudaStream_t stream);
cudaError_t launch_scan_decode(const ScanDecodeParams &p, cudaStream_t stream);
cudaError_t read_and_clear_scan_error(unsigned int *value);

// Steps of the forward that the backward takes too (kda_scan_fwd.cu): the states entering every
// cell of every sequence (states), and the gradients of the states leaving them (grads; what reaches a
// sequence's start goes to dh0). Cells (see scan_cells) lie on one grid over all tokens; sequence i's cell c has
// slot i + c of [slots, H, N, P]. `ws`: scan_states_workspace_bytes.
size_t scan_states_workspace_bytes(int64_t rows, int64_t n, int32_t H, int32_t P, int32_t N);
cudaError_t launch_scan_states(const ScanParams &p, float *states, float *grads, float *ws, cudaStream_t stream);

// On tcgen05 (kda_scan_tc.cu, kda_scan_tc_state.cu). The main run over pieces, state size 128, from the states in
// `entering` or from h0:
cudaError_t launch_scan_tc(const ScanParams &p, int64_t seg, int64_t units, const float *entering, cudaStream_t stream);
// and the state alone, with its weighted columns in 2 or 3 bf16 parts, over the tokens (fwd) and, with two
// directions, over dy and C backwards (rev).
struct ScanStateRun {
    const float *entering;   // the states that pieces enter with, or nullptr: h0 (dhT) where a sequence begins (ends)
    float *leave;            // what each piece adds, from zero, and its decay [pieces, H]; or nullptr
    float *leave_decay;
    float *states;           // the state at the entry (reverse: exit) of every cell of 128 tokens, or nullptr
};
cudaError_t launch_scan_tc_state(const ScanParams &p, int parts, int directions, int64_t seg, int64_t units,
                                 const ScanStateRun &fwd, const ScanStateRun &rev, cudaStream_t stream);
cudaError_t read_and_clear_scan_tc_error(unsigned int *value);
cudaError_t read_and_clear_scan_state_error(unsigned int *value);

constexpr int kScanTile = 64;     // tokens per tile
constexpr int kScanTcTile = 128;  // and of launch_scan_tc and the gradients
// The backward's tiles, and the cells that its states are kept for, are those of kScanTcTile. Slots of the cells of n
// sequences over `rows` tokens:
inline int64_t scan_cells(int64_t rows, int64_t n) { return rows / kScanTcTile + n; }

// The gradients of all tiles (kda_scan_tc_bwd.cu)
struct BwdWork {
    const float *states, *grads;   // [cells, H, N, P]: entering states, gradients of leaving states
    float *dbc;                    // [2][splits][rows][G][N] or nullptr (one split: written to dB, dC)
    float *part;                   // [cells][3][H]: sums of d dlog a, ddt, Q_tt
    int32_t splits;
    int64_t cells;
};
cudaError_t launch_scan_tc_bwd(const ScanParams &p, const BwdWork &w, cudaStream_t stream);
cudaError_t read_and_clear_scan_tc_bwd_error(unsigned int *value);

}  // namespace kda
