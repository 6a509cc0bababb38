// kda_scan_decode.cu -- one step of the selective scan (a single new token) for a batch of requests, sm_100a.
//
//   S <- a S + d B x^T,   y = S^T C + D x,   a = exp(d A), d = dt or softplus(dt + bias),
//
// for every request and head, with a state S of N x P. Bound by HBM: the state is read and written
// once (64 KiB of traffic per head at N = 128, P = 64 in fp32) against under 1 KiB of token vectors. One CTA
// per (request, head); a thread holds 16-byte pieces of the state's rows, all of whose loads are issued
// before anything is waited for. y adds up within the warp by shuffles and over warps in shared memory.
// Every element of the state is read and written by the same thread, so the step may run in place. (256 requests x
// 64 heads x 64 columns of 128, fp32, 1.08 GB: 160 us, 6.7 TB/s, a plain copy's rate.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_scan.cuh"

namespace kda {
namespace scan {

template <bool kFp32, int P, int N>
struct DecodeShape {
    static constexpr int E = kFp32 ? 4 : 8;              // elements per 16 bytes
    static constexpr int NT = kFp32 ? 256 : 128;         // bf16 states: half the bytes for the same fixed work
    static constexpr int LR = P / E;                     // threads per row of the state
    static constexpr int RP = NT / LR;                   // rows per pass
    static constexpr int PASSES = N / RP;
};

template <bool kFp32, int P, int N>
__global__ void __launch_bounds__(kFp32 ? 256 : 128) scan_decode_kernel(ScanDecodeParams p) {
    using L = DecodeShape<kFp32, P, N>;
    constexpr int E = L::E, NW = L::NT / 32;
    __shared__ float bs[N], cs[N], red[NW][P];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t bh = blockIdx.x, b = bh / p.H;
    const int h = static_cast<int>(bh - b * p.H);
    const int64_t st = bh * N * P;
    const int c0 = (tid % L::LR) * E, r0 = tid / L::LR;
    Vec<typename std::conditional<kFp32, float, __nv_bfloat16>::type, E> raw[L::PASSES];
#pragma unroll
    for (int k = 0; k < L::PASSES; ++k) {
        if (p.state_in)
            raw[k].load(p.state_in, st + static_cast<int64_t>(r0 + k * L::RP) * P + c0);
        else
            raw[k].zero();
    }
    const int64_t grp = h / (p.H / p.G);
    for (int n = tid; n < N; n += L::NT) {
        bs[n] = __uint_as_float(static_cast<uint32_t>(p.B[b * p.b_stride + grp * N + n]) << 16);
        cs[n] = __uint_as_float(static_cast<uint32_t>(p.C[b * p.c_stride + grp * N + n]) << 16);
    }
    float u;
    const float d = step_of(p.dt[bh], p.dt_bias ? p.dt_bias[h] : 0.f, p.softplus, &u);
    const float a = expf(d * p.A[h]);
    float xd[E], y[E];
    const uint16_t *x = p.x + b * p.x_stride + static_cast<int64_t>(h) * P;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        xd[e] = d * __uint_as_float(static_cast<uint32_t>(x[c0 + e]) << 16);
        y[e] = 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < L::PASSES; ++k) {
        const int r = r0 + k * L::RP;
        float s[E];
        raw[k].get(s);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            s[e] = fmaf(s[e], a, bs[r] * xd[e]);
            y[e] = fmaf(cs[r], s[e], y[e]);
        }
        if (p.state_out)
            Vec<typename std::conditional<kFp32, float, __nv_bfloat16>::type, E>::store(
                p.state_out, st + static_cast<int64_t>(r) * P + c0, s);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = L::LR; k < 32; k <<= 1) y[e] += __shfl_xor_sync(0xffffffffu, y[e], k);
    if (lane < L::LR)
#pragma unroll
        for (int e = 0; e < E; ++e) red[warp][c0 + e] = y[e];
    __syncthreads();
    const float Dh = p.D ? p.D[h] : 0.f;
    for (int c = 2 * tid; c < P; c += 2 * L::NT) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            s0 += red[w][c];
            s1 += red[w][c + 1];
        }
        const float x0 = __uint_as_float(static_cast<uint32_t>(x[c]) << 16);
        const float x1 = __uint_as_float(static_cast<uint32_t>(x[c + 1]) << 16);
        *reinterpret_cast<uint32_t *>(p.out + bh * P + c) = bf_pair(fmaf(Dh, x0, s0), fmaf(Dh, x1, s1));
    }
}

template <bool kFp32, int P, int N>
cudaError_t decode(const ScanDecodeParams &p, cudaStream_t s) {
    scan_decode_kernel<kFp32, P, N>
        <<<static_cast<unsigned>(p.batch * p.H), DecodeShape<kFp32, P, N>::NT, 0, s>>>(p);
    return cudaGetLastError();
}

template <bool kFp32>
cudaError_t decode(const ScanDecodeParams &p, cudaStream_t s) {
    if (p.P == 64) return p.N == 64 ? decode<kFp32, 64, 64>(p, s) : decode<kFp32, 64, 128>(p, s);
    return p.N == 64 ? decode<kFp32, 128, 64>(p, s) : decode<kFp32, 128, 128>(p, s);
}

}  // namespace scan

cudaError_t launch_scan_decode(const ScanDecodeParams &p, cudaStream_t s) {
    const int64_t units = p.batch * p.H;
    if (units <= 0) return cudaSuccess;
    if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return p.state_fp32 ? scan::decode<true>(p, s) : scan::decode<false>(p, s);
}

}  // namespace kda
