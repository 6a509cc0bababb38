// kda_scan_bwd.cu -- gradients of the selective state space scan, sm_100a.
//
// With a tile (128 tokens, entering state S_0, Gamma, L; see kda_scan_fwd.cu) and R the gradient of
// the state that leaves the tile, from the tokens behind it:
//
//   Q = dy x^T,   M = L . (C B^T),   K = L . Q Diag(d)
//   dx = Diag(d) M^T dy + Diag(d e^(Gamma_end - Gamma)) B R + D dy
//   dC = K B + Diag(e^Gamma) dy S_0^T
//   dB = K^T C + Diag(d e^(Gamma_end - Gamma)) x R^T                       (dB, dC: summed over a group's heads)
//   dd_s (through the input) = sum_t (M . Q)_ts + e^(Gamma_end - Gamma_s) B_s^T R x_s
//   dlog a_t = sum_{s < t <= u} (M . Q)_us d_s + sum_{u >= t} e^(Gamma_u) C_u^T S_0 dy_u
//              + sum_{s < t} d_s e^(Gamma_end - Gamma_s) B_s^T R x_s + e^(Gamma_end) <R, S_0>
//   ddelta = dd + A dlog a;   dA = sum d dlog a;   dD = sum_t Q_tt;   with softplus: ddt = ddelta sigmoid(dt + bias).
//
// Each pair (s, u) is counted in dlog a as it stands, never as a difference of sums over the whole
// sequence, so a long sequence loses no digits. C B^T and Q have operands that are exact in bf16, and M . Q
// is taken elementwise in fp32; the products with S_0 and R from which fp32 results follow take them as three
// bf16 parts (24 bits). M, K and the rows e^Gamma dy, d e^(Gamma_end - Gamma) x that multiply S_0^T, R^T (in two parts, 16
// bits) are rounded to bf16 once, for results in bf16.
//
// The states S_0 and gradients R of every tile come from two sweeps (launch_scan_states), fp32 in the
// workspace: that is its bulk. The gradient kernel (kda_scan_tc_bwd.cu) then takes all tiles at once. One CTA has one
// tile of one group and walks (a share of) the group's heads, so C B^T is computed once, and dB and dC add up over the
// heads on chip, without atomics. Where tiles x groups leave SMs idle the heads are shared out over several CTAs, whose
// dB and dC are added by scan_bc_kernel in a fixed order. Sums over tokens go by partial sums per tile, too: runs repeat
// bit for bit.
#include <cuda_runtime.h>

#include "kda_scan.cuh"

namespace kda {
namespace scan {

// dB and dC from the CTAs' shares, up to the last sequence's end; four values per thread
__global__ void __launch_bounds__(256) scan_bc_kernel(ScanParams p, BwdWork w) {
    const int64_t gn = static_cast<int64_t>(p.G) * p.N, plane = p.rows * gn;
    const int64_t e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (e >= plane) return;
    const int64_t row = e / gn;
    if (row >= p.seqs.end(p.seqs.n - 1)) return;
    const float *src = w.dbc + blockIdx.y * w.splits * plane + e;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < w.splits; ++k) {
        const float4 v = *reinterpret_cast<const float4 *>(src + k * plane);
        s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
    uint16_t *dst = blockIdx.y ? p.dC + row * p.dc_stride : p.dB + row * p.db_stride;
    *reinterpret_cast<uint2 *>(dst + (e - row * gn)) = make_uint2(bf_pair(s.x, s.y), bf_pair(s.z, s.w));
}

// dA, ddt_bias and dD from the tiles' sums: one CTA per head
__global__ void __launch_bounds__(256) scan_sum_kernel(ScanParams p, BwdWork w) {
    __shared__ double part[8];
    const int h = blockIdx.x, which = blockIdx.y;
    double s = 0;
    for (int64_t c = threadIdx.x; c < w.cells; c += 256) s += w.part[(c * 3 + which) * p.H + h];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i) s += part[i];
        float *dst = which == 0 ? p.dA : which == 1 ? p.ddt_bias : p.dD;
        if (dst) dst[h] = static_cast<float>(s);
    }
}

// CTAs that share a group's heads: the number that leaves the longest-working SM the fewest (tile, head)s, with one
// CTA per SM; the smallest such one, since each CTA's share of dB and dC is written and read again.
int head_splits(int64_t rows, int64_t n, int32_t H, int32_t G) {
    const int64_t ctas = scan_cells(rows, n) * G;
    const int per_group = H / G;
    int64_t best = 0;
    int best_s = 1;
    for (int s = 1; s <= per_group && s <= 32; ++s) {
        const int per = (per_group + s - 1) / s;
        if ((per_group + per - 1) / per != s) continue;   // a CTA without a head
        const int64_t cost = (ctas * s + 147) / 148 * (per + 1);   // what a CTA does once takes about a head's time
        if (s == 1 || cost < best) {
            best = cost;
            best_s = s;
        }
    }
    return best_s;
}

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

struct BwdLayout {
    size_t states, grads, dbc, part, pieces, total;   // byte offsets
    int splits;
};
BwdLayout bwd_layout(int64_t rows, int64_t n, int32_t H, int32_t G, int32_t P, int32_t N) {
    BwdLayout l;
    const size_t cells = static_cast<size_t>(scan_cells(rows, n));
    const size_t all = cells * H * N * P * sizeof(float);
    l.splits = head_splits(rows, n, H, G);
    l.states = 0;
    l.grads = round256(all);
    l.dbc = l.grads + round256(all);
    l.part = l.dbc + (l.splits > 1 ? round256(2 * static_cast<size_t>(l.splits) * rows * G * N * sizeof(float)) : 0);
    l.pieces = l.part + round256(cells * 3 * H * sizeof(float));
    l.total = l.pieces + round256(scan_states_workspace_bytes(rows, n, H, P, N));
    return l;
}

}  // namespace scan

size_t scan_bwd_workspace_bytes(int64_t rows, int64_t n, int32_t H, int32_t G, int32_t P, int32_t N) {
    return scan::bwd_layout(rows, n, H, G, P, N).total;
}

cudaError_t launch_scan_bwd(const ScanParams &p, cudaStream_t s) {
    using namespace scan;
    const BwdLayout l = bwd_layout(p.rows, p.seqs.n, p.H, p.G, p.P, p.N);
    uint8_t *ws = reinterpret_cast<uint8_t *>(p.ws);
    float *states = reinterpret_cast<float *>(ws + l.states), *grads = reinterpret_cast<float *>(ws + l.grads);
    float *pieces = reinterpret_cast<float *>(ws + l.pieces);
    BwdWork w;
    w.states = states;
    w.grads = grads;
    w.dbc = l.splits > 1 ? reinterpret_cast<float *>(ws + l.dbc) : nullptr;
    w.part = reinterpret_cast<float *>(ws + l.part);
    w.splits = l.splits;
    w.cells = scan_cells(p.rows, p.seqs.n);
    cudaError_t err = launch_scan_states(p, states, grads, pieces, s);
    if (err == cudaSuccess && w.cells > 0) err = launch_scan_tc_bwd(p, w, s);
    if (err == cudaSuccess && w.dbc && p.rows > 0) {
        const int64_t blocks = (p.rows * p.G * p.N / 4 + 255) / 256;
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
        scan_bc_kernel<<<dim3(static_cast<unsigned>(blocks), 2), 256, 0, s>>>(p, w);
        err = cudaGetLastError();
    }
    if (err == cudaSuccess) {
        scan_sum_kernel<<<dim3(static_cast<unsigned>(p.H), 3), 256, 0, s>>>(p, w);
        err = cudaGetLastError();
    }
    return err;
}

}  // namespace kda
