// kda_conv.cu -- short causal depthwise convolution with SiLU: prompts, gradients, single tokens. sm_100a.
//
// For every sequence, with e = [initial_state rows, x rows] (row -(W-1) .. -1 the state's):
//
//   pre_t = bias + sum_{k < W} w_k e_{t-W+1+k},   out_t = pre_t sigmoid(pre_t)  (or pre_t)
//
// All kernels are bound by HBM: 2 W operations and one sigmoid per element against 4 bytes
// (bf16, forward). A thread owns 4 channels (8 for single tokens) and walks a run of tokens with the
// last W - 1 inputs in registers, so x is read once but for the W - 1 rows before each run, which
// the neighbouring warp has just read. The loads of the next tokens are issued together, before any
// of them is used. Sums are fp32; each output is rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "kda_conv.h"

namespace kda {
namespace conv {

__device__ unsigned int g_conv_error = 0;

constexpr int V = 8;              // channels per thread, single tokens
constexpr int FV = 4;             // and forward: with 8 the taps and windows take twice the registers
constexpr int FW = 4;             // warps per CTA, forward
constexpr int U = 4;              // tokens of a batch
constexpr int kRing = 4;          // batches of loads in flight

// A thread's own window into shared memory for the rows it will need: asynchronous copies keep kRing batches of
// rows in flight without a register for any of them. Every thread reads back what it copied itself, so no
// barrier is needed. (71,000 tokens x 4096 bf16 channels: 200 us, 5.9 TB/s; with the rows 8 tokens ahead in
// registers 275 us.)
template <class T, int N, int kRows>
struct Ring {
    static constexpr int kBytes = N * sizeof(T);
    uint32_t at;    // this thread's place in row 0; rows are 32 * kBytes apart
    __device__ __forceinline__ uint32_t slot(int j) const {
        return at + static_cast<uint32_t>(j & (kRows - 1)) * (32 * kBytes);
    }
    __device__ __forceinline__ void copy(int j, const void *src, int64_t off) const {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(slot(j)),
                     "l"(static_cast<const T *>(src) + off), "n"(kBytes)
                     : "memory");
    }
    __device__ __forceinline__ void get(int j, float (&x)[N]) const {
        if constexpr (sizeof(T) == 4) {
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                         : "r"(slot(j)));
        } else {
            uint32_t a, b;
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(slot(j)));
            x[0] = bf_low(a);
            x[1] = bf_high(a);
            x[2] = bf_low(b);
            x[3] = bf_high(b);
        }
    }
};
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the `kLeft` youngest batches have arrived
template <int kLeft>
__device__ __forceinline__ void ring_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// 1 / (1 + e^-x) by the hardware's 2^y and 1/y (relative errors about 2^-22 each, and |x| 2^-24 of the rounding of 2^y's
// argument). With the flushing forms: those that keep denormals bring three times the instructions, which then bound the kernel.
__device__ __forceinline__ float sigmoidf(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

template <int W, int N>
__device__ __forceinline__ void load_taps(const ConvParams &p, int ch, float (&w)[W][N], float (&b)[N]) {
    // weight is [C, W]: the N channels' taps are N * W consecutive floats
    float flat[N * W];
    const float4 *src = reinterpret_cast<const float4 *>(p.weight + static_cast<int64_t>(ch) * W);
#pragma unroll
    for (int i = 0; i < N * W / 4; ++i) {
        const float4 f = src[i];
        flat[4 * i] = f.x;
        flat[4 * i + 1] = f.y;
        flat[4 * i + 2] = f.z;
        flat[4 * i + 3] = f.w;
    }
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int c = 0; c < N; ++c) w[k][c] = flat[c * W + k];
#pragma unroll
    for (int c = 0; c < N; ++c) b[c] = p.bias ? p.bias[ch + c] : 0.f;
}

// the row `back` tokens before row t of sequence i (which begins at b): of x, or of the initial state
template <class T, int W, int N>
__device__ __forceinline__ void load_before(const ConvParams &p, int32_t i, int64_t b, int64_t t, int back, int ch,
                                            float (&e)[N]) {
    Vec<T, N> raw;
    const int64_t pos = t - back - b;
    if (pos >= 0)
        raw.load(p.x, (t - back) * p.x_stride + ch);
    else if (p.init)
        raw.load(p.init, (static_cast<int64_t>(i) * (W - 1) + (W - 1) + pos) * p.C + ch);
    else
        raw.zero();
    raw.get(e);
}

// grid (token blocks + sequence blocks, channel blocks of 128). Token blocks: warp w walks `run` tokens.
// Sequence blocks: warp w copies the final state of one sequence.
template <class T, int W, bool kSilu>
__global__ void __launch_bounds__(32 * FW) conv_fwd_kernel(ConvParams p, int run, int64_t token_blocks) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ch = blockIdx.y * (32 * FV) + lane * FV;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seqs, &g_conv_error);
    if (blockIdx.x >= token_blocks) {
        const int64_t i64 = (static_cast<int64_t>(blockIdx.x) - token_blocks) * FW + warp;
        if (i64 >= p.seqs.n || ch >= p.C) return;
        const int32_t i = static_cast<int32_t>(i64);
        const int64_t b = p.seqs.begin(i), e = p.seqs.end(i);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float f[FV];
            load_before<T, W, FV>(p, i, b, e, W - 1 - k, ch, f);
            Vec<T, FV>::store(p.final_state, (i64 * (W - 1) + k) * p.C + ch, f);
        }
        return;
    }
    int64_t t = (static_cast<int64_t>(blockIdx.x) * FW + warp) * run;
    if (t >= p.rows) return;
    const int64_t t1 = t + run < p.rows ? t + run : p.rows;
    int32_t i = warp_upper(p.seqs.n, t, [&](int32_t j) { return p.seqs.begin(j); });
    int64_t b = p.seqs.begin(i), e = p.seqs.end(i);
    if (ch >= p.C) return;
    float w[W][FV], bias[FV];
    load_taps<W, FV>(p, ch, w, bias);
    __shared__ __align__(16) uint8_t rows_s[FW][kRing * U * 32 * FV * sizeof(T)];
    const Ring<T, FV, kRing * U> ring = {static_cast<uint32_t>(__cvta_generic_to_shared(rows_s[warp])) +
                                     static_cast<uint32_t>(lane * FV * sizeof(T))};
    const int n = static_cast<int>(t1 - t);
    const int64_t x0 = t * p.x_stride + ch;
    auto fetch = [&](int j) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u < n) ring.copy(j + u, p.x, x0 + (j + u) * p.x_stride);
        ring_commit();
    };
    for (int k = 0; k < kRing - 1; ++k) fetch(k * U);
    float win[W - 1][FV];
    int64_t yi = t * p.out_stride + ch;
    // tokens of sequence i from the run's start; the next sequence with tokens
    int left = 0;
    auto enter = [&](int j) {
        while (t + j >= e) {
            if (++i >= p.seqs.n) return false;   // behind the last sequence nothing is written
            b = p.seqs.begin(i);
            e = p.seqs.end(i);
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) load_before<T, W, FV>(p, i, b, t + j, W - 1 - k, ch, win[k]);
        left = static_cast<int>(e - t < n ? e - t : n);
        return true;
    };
    if (!enter(0)) return;
    auto step = [&](int j) {
        float x[FV], y[FV];
        ring.get(j, x);
#pragma unroll
        for (int c = 0; c < FV; ++c) {
            float a = fmaf(w[W - 1][c], x[c], bias[c]);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) a = fmaf(w[k][c], win[k][c], a);
            y[c] = kSilu ? a * sigmoidf(a) : a;
#pragma unroll
            for (int k = 0; k < W - 2; ++k) win[k][c] = win[k + 1][c];
            win[W - 2][c] = x[c];
        }
        Vec<T, FV>::store(p.out, yi, y);
        yi += p.out_stride;
    };
    for (int j = 0; j < n; j += U) {
        fetch(j + (kRing - 1) * U);
        ring_wait<kRing - 1>();
        if (j + U <= left) {
#pragma unroll
            for (int u = 0; u < U; ++u) step(j + u);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (j + u >= n) break;
                if (j + u >= left && !enter(j + u)) return;
                step(j + u);
            }
        }
    }
}

// ---------------------------------------------------------------- single tokens

// A thread takes kRows requests of its 8 channels, with the taps read once: at 256 x 12288 bf16 the taps alone, read
// for every request, were as many bytes again as everything else (20 us; with four requests 9.0, 5.6 TB/s).
template <class T, int W, bool kSilu, int kRows>
__global__ void __launch_bounds__(128) conv_decode_kernel(ConvDecodeParams p) {
    const int ch = (blockIdx.x * 128 + threadIdx.x) * V;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kRows;
    if (ch >= p.C) return;
    Vec<T, V> x[kRows], s[kRows][W - 1];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (r0 + r >= p.batch) break;
        x[r].load(p.x, (r0 + r) * p.x_stride + ch);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            if (p.state_in)
                s[r][k].load(p.state_in, ((r0 + r) * (W - 1) + k) * p.C + ch);
            else
                s[r][k].zero();
        }
    }
    ConvParams tp;
    tp.weight = p.weight;
    tp.bias = p.bias;
    float w[W][V], bias[V];
    load_taps<W, V>(tp, ch, w, bias);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (r0 + r >= p.batch) break;
        const int64_t st = (r0 + r) * (W - 1) * p.C + ch;
        float f[V], y[V];
        x[r].get(f);
#pragma unroll
        for (int c = 0; c < V; ++c) y[c] = fmaf(w[W - 1][c], f[c], bias[c]);
        if (p.state_out) Vec<T, V>::store(p.state_out, st + static_cast<int64_t>(W - 2) * p.C, f);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            s[r][k].get(f);
#pragma unroll
            for (int c = 0; c < V; ++c) y[c] = fmaf(w[k][c], f[c], y[c]);
            // in place: the thread has read all its rows of the state before it writes any
            if (k > 0 && p.state_out) Vec<T, V>::store(p.state_out, st + static_cast<int64_t>(k - 1) * p.C, f);
        }
        if (kSilu)
#pragma unroll
            for (int c = 0; c < V; ++c) y[c] *= sigmoidf(y[c]);
        Vec<T, V>::store(p.out, (r0 + r) * p.out_stride + ch, y);
    }
}

// ---------------------------------------------------------------- gradients
//
//   dpre_t = dout_t act'(pre_t)  with pre recomputed from x,
//   de_j = sum_k w_k dpre_{j+W-1-k} (outputs of the same sequence) + dfinal_state,
//   dw_k = sum_t dpre_t e_{t-W+1+k},  dbias = sum_t dpre_t.
//
// A warp walks one run of tokens and the W - 1 behind them (whose dpre it needs for its last dx). 4 channels
// per thread keep the taps, their gradients and both windows within 128 registers. Each CTA adds its
// warps' tap gradients in shared memory and writes one partial row; conv_reduce_kernel adds the rows
// in a fixed order, so a run repeats bit for bit.

constexpr int BV = 4;             // channels per thread
constexpr int kBwdRing = 2;       // batches in flight, of four tokens (fp32: two)
constexpr int BW = 8;             // warps per CTA
constexpr int kMinRun = 32;       // tokens per warp, at least

template <int W, bool kSilu>
__device__ __forceinline__ void dpre_of(const float (&w)[W][BV], const float (&bias)[BV], const float (&win)[W - 1][BV],
                                        const float (&x)[BV], const float (&dy)[BV], float (&d)[BV]) {
#pragma unroll
    for (int c = 0; c < BV; ++c) {
        d[c] = dy[c];
        if (kSilu) {
            float a = fmaf(w[W - 1][c], x[c], bias[c]);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) a = fmaf(w[k][c], win[k][c], a);
            const float g = sigmoidf(a);
            d[c] *= g * fmaf(a, 1.f - g, 1.f);
        }
    }
}

// grid (token blocks + sequence blocks, channel blocks of 128). Sequence blocks write dinit: warp w one
// sequence.
template <class T, class TD, int W, bool kSilu>
__global__ void __launch_bounds__(32 * BW, 2) conv_bwd_kernel(ConvParams p, int token_blocks, int64_t run) {
    // the rings, and when they are done with, the warps' sums
    constexpr int BU = sizeof(T) == 4 ? 2 : 4;
    constexpr int kX = kBwdRing * BU * 32 * BV * sizeof(T), kD = kBwdRing * BU * 32 * BV * sizeof(TD);
    constexpr int kPart = (W + 1) * 32 * BV * sizeof(float), kWarp = kX + kD > kPart ? kX + kD : kPart;
    __shared__ __align__(16) uint8_t shared[BW * kWarp];
    float(*part)[W + 1][32 * BV] = reinterpret_cast<float(*)[W + 1][32 * BV]>(shared);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ch = blockIdx.y * (32 * BV) + lane * BV;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seqs, &g_conv_error);
    float w[W][BV], bias[BV];
    if (ch < p.C) load_taps<W, BV>(p, ch, w, bias);
    if (blockIdx.x >= token_blocks) {
        // de_j for the rows before the sequence: its first W - 1 outputs, and what a sequence shorter
        // than the state passes on from the final state's gradient
        const int64_t i64 = (static_cast<int64_t>(blockIdx.x) - token_blocks) * BW + warp;
        if (i64 >= p.seqs.n || ch >= p.C) return;
        const int32_t i = static_cast<int32_t>(i64);
        const int64_t b = p.seqs.begin(i), e = p.seqs.end(i);
        float de[W - 1][BV], win[W - 1][BV];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            load_before<T, W, BV>(p, i, b, b, W - 1 - j, ch, win[j]);
            const int64_t slot = j - (e - b);
            if (p.dfinal && slot >= 0) {
                Vec<T, BV> r;
                r.load(p.dfinal, (i64 * (W - 1) + slot) * p.C + ch);
                r.get(de[j]);
            } else {
#pragma unroll
                for (int c = 0; c < BV; ++c) de[j][c] = 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < W - 1; ++u) {
            if (b + u < e) {
                Vec<T, BV> rx;
                Vec<TD, BV> rd;
                float x[BV], dy[BV], d[BV];
                rx.load(p.x, (b + u) * p.x_stride + ch);
                rd.load(p.dout, (b + u) * p.dout_stride + ch);
                rx.get(x);
                rd.get(dy);
                dpre_of<W, kSilu>(w, bias, win, x, dy, d);
                // output u reads row j of the state (place j - (W - 1)) with tap j - u
#pragma unroll
                for (int j = u; j < W - 1; ++j)
#pragma unroll
                    for (int c = 0; c < BV; ++c) de[j][c] = fmaf(w[j - u][c], d[c], de[j][c]);
#pragma unroll
                for (int c = 0; c < BV; ++c) {
#pragma unroll
                    for (int k = 0; k < W - 2; ++k) win[k][c] = win[k + 1][c];
                    win[W - 2][c] = x[c];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) Vec<T, BV>::store(p.dinit, (i64 * (W - 1) + j) * p.C + ch, de[j]);
        return;
    }
    float dw[W + 1][BV];
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int c = 0; c < BV; ++c) dw[k][c] = 0.f;
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(shared)) + warp * kWarp;
    const Ring<T, BV, kBwdRing * BU> x_ring = {mine + static_cast<uint32_t>(lane * BV * sizeof(T))};
    const Ring<TD, BV, kBwdRing * BU> d_ring = {mine + kX + static_cast<uint32_t>(lane * BV * sizeof(TD))};
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * BW + warp) * run;
    if (t0 < p.rows) {
        const int64_t t1 = t0 + run < p.rows ? t0 + run : p.rows;
        int32_t i = warp_upper(p.seqs.n, t0, [&](int32_t j) { return p.seqs.begin(j); });
        int64_t a = ch < p.C ? t0 : t1;
        while (a < t1) {
            // the part [a, z) of the run that belongs to sequence i = [b, e)
            int64_t b = p.seqs.begin(i), e = p.seqs.end(i);
            while (a >= e && i + 1 < p.seqs.n) {
                ++i;
                b = p.seqs.begin(i);
                e = p.seqs.end(i);
            }
            if (a >= e) break;   // rows behind the last sequence
            const int64_t z = t1 < e ? t1 : e;
            float win[W - 1][BV], dp[W - 1][BV];
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                load_before<T, W, BV>(p, i, b, a, W - 1 - k, ch, win[k]);
#pragma unroll
                for (int c = 0; c < BV; ++c) dp[k][c] = 0.f;
            }
            // counted from a: outputs n (own), tokens of the sequence left (up to the W - 1 behind the run), steps,
            // and the first token whose place the final state holds
            const int n = static_cast<int>(z - a), left = static_cast<int>(e - a < n + W - 1 ? e - a : n + W - 1);
            const int steps = n + W - 1, kept = p.dfinal && e - a <= n + W - 1 ? static_cast<int>(e - a) - (W - 1) : n;
            int64_t xi = a * p.x_stride + ch, di = a * p.dout_stride + ch;
            int64_t oi = (a - (W - 1)) * p.dx_stride + ch;
            auto fetch = [&](int j) {
#pragma unroll
                for (int u = 0; u < BU; ++u) {
                    if (j + u < left) {
                        x_ring.copy(j + u, p.x, xi + (j + u) * p.x_stride);
                        d_ring.copy(j + u, p.dout, di + (j + u) * p.dout_stride);
                    }
                }
                ring_commit();
            };
            // step j: dpre of token a + j, and with it dx of token a + j - (W - 1). kInner: all of that is there
            auto step = [&](auto inner, int j) {
                constexpr bool kInner = decltype(inner)::value;
                float x[BV], dy[BV], d[BV];
                if (kInner || j < left) {
                    x_ring.get(j, x);
                    d_ring.get(j, dy);
                    dpre_of<W, kSilu>(w, bias, win, x, dy, d);
                } else {
#pragma unroll
                    for (int c = 0; c < BV; ++c) x[c] = d[c] = 0.f;   // behind the sequence
                }
                if (kInner || j >= W - 1) {
                    float g[BV];
#pragma unroll
                    for (int c = 0; c < BV; ++c) {
                        g[c] = w[0][c] * d[c];
#pragma unroll
                        for (int k = 1; k < W; ++k) g[c] = fmaf(w[k][c], dp[W - 1 - k][c], g[c]);
                    }
                    const int o = j - (W - 1);
                    if (!kInner && o >= kept) {
                        Vec<T, BV> r;
                        float f[BV];
                        r.load(p.dfinal, (static_cast<int64_t>(i) * (W - 1) + o + (W - 1) - (e - a)) * p.C + ch);
                        r.get(f);
#pragma unroll
                        for (int c = 0; c < BV; ++c) g[c] += f[c];
                    }
                    Vec<T, BV>::store(p.dx, oi, g);
                }
                oi += p.dx_stride;
                if (kInner || j < n) {
#pragma unroll
                    for (int c = 0; c < BV; ++c) {
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) dw[k][c] = fmaf(d[c], win[k][c], dw[k][c]);
                        dw[W - 1][c] = fmaf(d[c], x[c], dw[W - 1][c]);
                        dw[W][c] += d[c];
                    }
                }
#pragma unroll
                for (int c = 0; c < BV; ++c) {
#pragma unroll
                    for (int k = 0; k < W - 2; ++k) {
                        win[k][c] = win[k + 1][c];
                        dp[k][c] = dp[k + 1][c];
                    }
                    win[W - 2][c] = x[c];
                    dp[W - 2][c] = d[c];
                }
            };
            for (int k = 0; k < kBwdRing - 1; ++k) fetch(k * BU);
            for (int j = 0; j < steps; j += BU) {
                fetch(j + (kBwdRing - 1) * BU);
                ring_wait<kBwdRing - 1>();
                if (j >= W - 1 && j + BU <= n && j + BU - (W - 1) <= kept) {
#pragma unroll
                    for (int u = 0; u < BU; ++u) step(std::true_type(), j + u);
                } else {
#pragma unroll
                    for (int u = 0; u < BU; ++u)
                        if (j + u < steps) step(std::false_type(), j + u);
                }
            }
            ring_wait<0>();
            a = z;
        }
    }
    __syncthreads();   // every warp is done with its rings
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int c = 0; c < BV; ++c) part[warp][k][lane * BV + c] = dw[k][c];
    __syncthreads();
    for (int j = threadIdx.x; j < (W + 1) * 32 * BV; j += 32 * BW) {
        const int k = j / (32 * BV), c = j % (32 * BV), gc = blockIdx.y * (32 * BV) + c;
        if (gc >= p.C) continue;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < BW; ++q) s += part[q][k][c];
        p.partial[(static_cast<int64_t>(blockIdx.x) * (W + 1) + k) * p.C + gc] = s;
    }
}

template <int W>
__global__ void __launch_bounds__(128) conv_reduce_kernel(ConvParams p, int blocks) {
    const int c = blockIdx.x * 128 + threadIdx.x, k = blockIdx.y;
    if (c >= p.C) return;
    float s = 0.f;
#pragma unroll 4
    for (int b = 0; b < blocks; ++b) s += p.partial[(static_cast<int64_t>(b) * (W + 1) + k) * p.C + c];
    if (k < W) {
        if (p.dweight) p.dweight[static_cast<int64_t>(c) * W + k] = s;
    } else if (p.dbias) {
        p.dbias[c] = s;
    }
}

template <class F>
cudaError_t by_taps(int W, F f) {
    switch (W) {
        case 2: return f(std::integral_constant<int, 2>());
        case 3: return f(std::integral_constant<int, 3>());
        default: return f(std::integral_constant<int, 4>());
    }
}

template <class T, int W>
cudaError_t fwd(const ConvParams &p, cudaStream_t s) {
    // Long runs re-read fewer rows (W - 1 of every `run`); short ones make enough warps of few tokens.
    const int64_t cblocks = (p.C + 32 * FV - 1) / (32 * FV);
    int run = 64;
    while (run > U && (p.rows + run - 1) / run * cblocks < 148 * 32) run /= 2;
    const int64_t tb = (p.rows + FW * run - 1) / (FW * run);
    const int64_t sb = p.final_state ? (p.seqs.n + FW - 1) / FW : 0;
    if (tb + sb == 0) return cudaSuccess;
    if (tb + sb > 0x7fffffffLL || cblocks > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(tb + sb), static_cast<unsigned>(cblocks));
    if (p.silu)
        conv_fwd_kernel<T, W, true><<<grid, 32 * FW, 0, s>>>(p, run, tb);
    else
        conv_fwd_kernel<T, W, false><<<grid, 32 * FW, 0, s>>>(p, run, tb);
    return cudaGetLastError();
}

template <class T, class TD, int W>
cudaError_t bwd(const ConvParams &p, cudaStream_t s) {
    const int32_t tb = conv_bwd_blocks(p.rows, p.C);
    const int64_t cblocks = (p.C + 32 * BV - 1) / (32 * BV);
    const int64_t sb = p.dinit ? (p.seqs.n + BW - 1) / BW : 0, run = (p.rows + tb * BW - 1) / (tb * BW);
    if (tb + sb > 0x7fffffffLL || cblocks > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(tb + sb), static_cast<unsigned>(cblocks));
    if (p.silu)
        conv_bwd_kernel<T, TD, W, true><<<grid, 32 * BW, 0, s>>>(p, tb, run);
    else
        conv_bwd_kernel<T, TD, W, false><<<grid, 32 * BW, 0, s>>>(p, tb, run);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || (!p.dweight && !p.dbias)) return err;
    conv_reduce_kernel<W><<<dim3((p.C + 127) / 128, W + 1), 128, 0, s>>>(p, tb);
    return cudaGetLastError();
}

template <class T, int W, int kRows>
cudaError_t decode(const ConvDecodeParams &p, cudaStream_t s) {
    const int64_t y = (p.batch + kRows - 1) / kRows;
    const dim3 grid(static_cast<unsigned>((p.C / V + 127) / 128), static_cast<unsigned>(y));
    if (p.silu)
        conv_decode_kernel<T, W, true, kRows><<<grid, 128, 0, s>>>(p);
    else
        conv_decode_kernel<T, W, false, kRows><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

template <class T, int W>
cudaError_t decode(const ConvDecodeParams &p, cudaStream_t s) {
    // four requests per thread where that leaves eight warps per SM, and always beyond what one grid holds
    if (p.batch * (p.C / V) >= 4 * 148 * 256 || p.batch > 65535) {
        if ((p.batch + 3) / 4 > 65535) {
            // more than 262140 requests: one launch for each so many
            for (int64_t r = 0; r < p.batch; r += 4 * 65535) {
                ConvDecodeParams q = p;
                const int64_t e = sizeof(T), st = r * (W - 1) * p.C * e;
                q.batch = p.batch - r < 4 * 65535 ? p.batch - r : 4 * 65535;
                q.x = static_cast<const uint8_t *>(p.x) + r * p.x_stride * e;
                q.out = static_cast<uint8_t *>(p.out) + r * p.out_stride * e;
                q.state_in = p.state_in ? static_cast<const uint8_t *>(p.state_in) + st : nullptr;
                q.state_out = p.state_out ? static_cast<uint8_t *>(p.state_out) + st : nullptr;
                const cudaError_t err = decode<T, W, 4>(q, s);
                if (err != cudaSuccess) return err;
            }
            return cudaSuccess;
        }
        return decode<T, W, 4>(p, s);
    }
    return decode<T, W, 1>(p, s);
}

}  // namespace conv

int32_t conv_bwd_blocks(int64_t rows, int32_t C) {
    // one round of two CTAs per SM over all channel blocks: each writes one row of partial sums
    const int64_t cblocks = (static_cast<int64_t>(C) + 32 * conv::BV - 1) / (32 * conv::BV);
    const int64_t most = (rows + conv::BW * conv::kMinRun - 1) / (conv::BW * conv::kMinRun);
    const int64_t want = 2 * 148 / cblocks;
    const int64_t n = most < want ? most : want;
    return static_cast<int32_t>(n < 1 ? 1 : n);
}

cudaError_t launch_conv_fwd(const ConvParams &p, cudaStream_t s) {
    return conv::by_taps(p.W, [&](auto w) {
        constexpr int W = decltype(w)::value;
        return p.fp32 ? conv::fwd<float, W>(p, s) : conv::fwd<__nv_bfloat16, W>(p, s);
    });
}

cudaError_t launch_conv_bwd(const ConvParams &p, cudaStream_t s) {
    return conv::by_taps(p.W, [&](auto w) {
        constexpr int W = decltype(w)::value;
        if (p.fp32) return conv::bwd<float, float, W>(p, s);
        return p.dout_fp32 ? conv::bwd<__nv_bfloat16, float, W>(p, s) : conv::bwd<__nv_bfloat16, __nv_bfloat16, W>(p, s);
    });
}

cudaError_t launch_conv_decode(const ConvDecodeParams &p, cudaStream_t s) {
    return conv::by_taps(p.W, [&](auto w) {
        constexpr int W = decltype(w)::value;
        return p.fp32 ? conv::decode<float, W>(p, s) : conv::decode<__nv_bfloat16, W>(p, s);
    });
}

cudaError_t read_and_clear_conv_error(unsigned int *value) {
    cudaError_t err = cudaMemcpyFromSymbol(value, conv::g_conv_error, sizeof(*value));
    if (err != cudaSuccess || *value == 0) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(conv::g_conv_error, &zero, sizeof(zero));
}

}  // namespace kda
