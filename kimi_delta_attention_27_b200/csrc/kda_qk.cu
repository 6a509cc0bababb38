// kda_qk.cu -- per-head norm of queries and keys and their position rotation in one pass, and its gradient. sm_100a.
//
// For each token and head, with x the head's D channels:
//
//   r = (sum x^2 + eps)^(-1/2) (L2), (mean x^2 + eps)^(-1/2) (RMS) or 1;   z = x r w
//   (z_i, z_j) -> (z_i cos - z_j sin, z_j cos + z_i sin) for the pairs of the first `rot` channels,
//
// pairs (2i, 2i + 1) or (i, i + rot / 2), angle position * inv_freq_i, cos and sin times `factor`.
//
// Bound by HBM: 4 bytes per channel against some 20 operations. D / 8 lanes hold a head, 8 channels each
// (16-byte accesses), so a warp takes 256 / D heads at a time; sums and the half layout's partners go by
// shuffles within the head's lanes. A warp walks the heads of one token: its lanes' angles are computed
// once, while the first loads are in flight, and serve all of them. Few tokens: several warps share one.
//
// An angle can be 10^6 radians, where 32 bits are off by 0.06: position * inv_freq is formed and reduced to a
// fraction of a turn in 64 bits, which is then exact enough in 32 (2^-25 of a turn).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_qk.h"
#include "kda_seq.cuh"

namespace kda {
namespace qk {

constexpr int V = 8;              // channels per lane
constexpr int NW = 8;             // warps per CTA
constexpr int U = 4;              // passes whose loads are issued together

// the lane's rotation: cos and sin of its channels' pairs (sin with the sign that the channel needs)
struct Turn {
    float c[V], s[V];
};

__device__ __forceinline__ void angle(const QkParams &p, double pos, int i, float *c, float *s) {
    const double turns = pos * (static_cast<double>(p.inv_freq[i]) * 0.15915494309189533577);
    const float f = static_cast<float>(turns - rint(turns));
    sincospif(2.f * f, s, c);
    *c *= p.factor;
    *s *= p.factor;
}

// sign: 1 forward, -1 for the transposed rotation
__device__ __forceinline__ void make_turn(const QkParams &p, int64_t row, int c0, float sign, Turn &t) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        t.c[j] = 1.f;
        t.s[j] = 0.f;
    }
    if (c0 >= p.rot) return;
    const double pos = static_cast<double>(p.positions[row]);
    if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            float c, s;
            angle(p, pos, (c0 + j) >> 1, &c, &s);
            t.c[j] = t.c[j + 1] = c;
            t.s[j] = -sign * s;
            t.s[j + 1] = sign * s;
        }
    } else {
        const int half = p.rot >> 1;
        const bool low = c0 < half;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float c, s;
            angle(p, pos, (low ? c0 : c0 - half) + j, &c, &s);
            t.c[j] = c;
            t.s[j] = low ? -sign * s : sign * s;
        }
    }
}

// z rotated in place: z_i c_i + z_partner(i) s_i
__device__ __forceinline__ void rotate(const QkParams &p, const Turn &t, int c0, float (&z)[V]) {
    if (p.rot == 0) return;
    if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const float a = z[j], b = z[j + 1];
            z[j] = fmaf(a, t.c[j], b * t.s[j]);
            z[j + 1] = fmaf(b, t.c[j + 1], a * t.s[j + 1]);
        }
    } else {
        const int lane = threadIdx.x & 31, by = p.rot >> 4;   // rot / 2 channels are rot / 16 lanes
        const int from = c0 >= p.rot ? lane : (2 * c0 < p.rot ? lane + by : lane - by);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float b = __shfl_sync(0xffffffffu, z[j], from);
            z[j] = fmaf(z[j], t.c[j], b * t.s[j]);
        }
    }
}

template <int LPH>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
    for (int d = LPH / 2; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// 1 / norm; a zero vector without eps stays zero
template <int D>
__device__ __forceinline__ float inverse_norm(const QkParams &p, const float (&x)[V]) {
    if (p.norm == kNormNone) return 1.f;   // the same for all lanes
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) ss = fmaf(x[j], x[j], ss);
    ss = head_sum<D / V>(ss);
    if (p.norm == kNormRms) ss *= 1.f / D;
    ss += p.eps;
    return ss == 0.f ? 0.f : rsqrtf(ss);
}

template <int D>
__global__ void __launch_bounds__(32 * NW) qk_fwd_kernel(QkParams p, int per_token) {
    constexpr int LPH = D / V, HPW = 32 / LPH;
    const int lane = threadIdx.x & 31, c0 = (lane % LPH) * V, sub = lane / LPH;
    const int64_t task = static_cast<int64_t>(blockIdx.x) * NW + (threadIdx.x >> 5);
    const int64_t row = task / per_token;
    if (row >= p.rows) return;
    const int heads = p.Hq + p.Hk, step = per_token * HPW;
    const int first = static_cast<int>(task - row * per_token) * HPW;
    Turn t;
    float wq[V], wk[V];
    bool ready = false;
    for (int h0 = first; h0 < heads; h0 += U * step) {
        Vec<__nv_bfloat16, V> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * step + sub;
            if (h < p.Hq)
                raw[u].load(p.q, row * p.q_stride + static_cast<int64_t>(h) * D + c0);
            else if (h < heads)
                raw[u].load(p.k, row * p.k_stride + static_cast<int64_t>(h - p.Hq) * D + c0);
            else
                raw[u].zero();
        }
        if (!ready) {
            ready = true;
            make_turn(p, row, c0, 1.f, t);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                wq[j] = p.q_weight ? p.q_weight[c0 + j] : 1.f;
                wk[j] = p.k_weight ? p.k_weight[c0 + j] : 1.f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h0 + u * step >= heads) break;   // the same for the warp
            const int h = h0 + u * step + sub;
            float z[V];
            raw[u].get(z);
            const float r = inverse_norm<D>(p, z);
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] *= r * (h < p.Hq ? wq[j] : wk[j]);
            rotate(p, t, c0, z);
            if (h < p.Hq)
                Vec<__nv_bfloat16, V>::store(p.q_out, row * p.q_out_stride + static_cast<int64_t>(h) * D + c0, z);
            else if (h < heads)
                Vec<__nv_bfloat16, V>::store(p.k_out, row * p.k_out_stride + static_cast<int64_t>(h - p.Hq) * D + c0,
                                             z);
        }
    }
}

// Gradients: dz is the rotation's transpose applied to the given gradient,
//   dx = r (w dz - xh <xh, w dz> / (1 or D)),  xh = x r,   dw = sum over tokens and heads of dz xh.
// CTAs walk the tasks, so that there are few partial sums of dw; they are added in a fixed order.
template <int D, class TD>
__global__ void __launch_bounds__(32 * NW) qk_bwd_kernel(QkParams p, int per_token, int64_t tasks) {
    constexpr int LPH = D / V, HPW = 32 / LPH, UB = 2;
    __shared__ float part[NW][HPW][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = (lane % LPH) * V, sub = lane / LPH;
    const int heads = p.Hq + p.Hk, step = per_token * HPW;
    float wq[V], wk[V], dwq[V], dwk[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        wq[j] = p.q_weight ? p.q_weight[c0 + j] : 1.f;
        wk[j] = p.k_weight ? p.k_weight[c0 + j] : 1.f;
        dwq[j] = dwk[j] = 0.f;
    }
    const float share = p.norm == kNormRms ? 1.f / D : 1.f;
    for (int64_t task = static_cast<int64_t>(blockIdx.x) * NW + warp; task < tasks;
         task += static_cast<int64_t>(gridDim.x) * NW) {
        const int64_t row = task / per_token;
        const int first = static_cast<int>(task - row * per_token) * HPW;
        Turn t;
        bool ready = false;
        for (int h0 = first; h0 < heads; h0 += UB * step) {
            Vec<__nv_bfloat16, V> rx[UB];
            Vec<TD, V> rd[UB];
#pragma unroll
            for (int u = 0; u < UB; ++u) {
                const int h = h0 + u * step + sub;
                if (h < p.Hq) {
                    rx[u].load(p.q, row * p.q_stride + static_cast<int64_t>(h) * D + c0);
                    rd[u].load(p.dq_out, row * p.dq_stride + static_cast<int64_t>(h) * D + c0);
                } else if (h < heads) {
                    rx[u].load(p.k, row * p.k_stride + static_cast<int64_t>(h - p.Hq) * D + c0);
                    rd[u].load(p.dk_out, row * p.dk_stride + static_cast<int64_t>(h - p.Hq) * D + c0);
                } else {
                    rx[u].zero();
                    rd[u].zero();
                }
            }
            if (!ready) {
                ready = true;
                make_turn(p, row, c0, -1.f, t);
            }
#pragma unroll
            for (int u = 0; u < UB; ++u) {
                if (h0 + u * step >= heads) break;
                const int h = h0 + u * step + sub;
                const bool is_q = h < p.Hq;
                float x[V], d[V];
                rx[u].get(x);
                rd[u].get(d);
                rotate(p, t, c0, d);
                if (p.norm != kNormNone) {
                    const float r = inverse_norm<D>(p, x);
                    float dot = 0.f;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        x[j] *= r;
                        const float g = d[j] * x[j];
                        if (is_q)
                            dwq[j] += g;
                        else
                            dwk[j] += g;
                        const float w = is_q ? wq[j] : wk[j];
                        dot = fmaf(g, w, dot);
                        d[j] *= w;
                    }
                    dot = head_sum<LPH>(dot) * share;
#pragma unroll
                    for (int j = 0; j < V; ++j) d[j] = r * fmaf(-x[j], dot, d[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float g = d[j] * x[j];
                        if (is_q)
                            dwq[j] += g;
                        else
                            dwk[j] += g;
                        d[j] *= is_q ? wq[j] : wk[j];
                    }
                }
                if (is_q)
                    Vec<__nv_bfloat16, V>::store(p.q_out, row * p.q_out_stride + static_cast<int64_t>(h) * D + c0, d);
                else if (h < heads)
                    Vec<__nv_bfloat16, V>::store(p.k_out,
                                                 row * p.k_out_stride + static_cast<int64_t>(h - p.Hq) * D + c0, d);
            }
        }
    }
    if (!p.partial) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) part[warp][sub][c0 + j] = which ? dwk[j] : dwq[j];
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += 32 * NW) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w)
#pragma unroll
                for (int q = 0; q < HPW; ++q) s += part[w][q][c];
            p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + which) * D + c] = s;
        }
    }
}

// grid 2 D / 32: 32 sums per CTA, 8 threads each
__global__ void __launch_bounds__(256) qk_reduce_kernel(QkParams p, int blocks) {
    __shared__ float part[8][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, at = blockIdx.x * 32 + x;
    float s = 0.f;
#pragma unroll 4
    for (int b = y; b < blocks; b += 8) s += p.partial[static_cast<int64_t>(b) * 2 * p.D + at];
    part[y][x] = s;
    __syncthreads();
    if (y == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][x];
        if (at < p.D) {
            if (p.dq_weight) p.dq_weight[at] = s;
        } else if (p.dk_weight) {
            p.dk_weight[at - p.D] = s;
        }
    }
}

// warps per token: one where that makes 16 warps per SM, else as many as it takes, up to one per pass
int warps_per_token(int64_t rows, int32_t heads, int32_t D) {
    const int passes = (heads * D + 255) / 256;
    int n = 1;
    while (n < passes && rows * n < 148 * 16) n *= 2;
    return n < passes ? n : passes;
}

template <class F>
cudaError_t by_dim(int D, F f) {
    switch (D) {
        case 64: return f(std::integral_constant<int, 64>());
        case 128: return f(std::integral_constant<int, 128>());
        default: return f(std::integral_constant<int, 256>());
    }
}

}  // namespace qk

int32_t qk_bwd_blocks(int64_t rows, int32_t heads, int32_t D) {
    const int64_t tasks = rows * qk::warps_per_token(rows, heads, D);
    const int64_t n = (tasks + qk::NW - 1) / qk::NW;
    return static_cast<int32_t>(n < 1 ? 1 : (n < 4 * 148 ? n : 4 * 148));
}

cudaError_t launch_qk_fwd(const QkParams &p, cudaStream_t s) {
    if (p.rows == 0) return cudaSuccess;
    const int per = qk::warps_per_token(p.rows, p.Hq + p.Hk, p.D);
    const int64_t blocks = (p.rows * per + qk::NW - 1) / qk::NW;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return qk::by_dim(p.D, [&](auto d) {
        qk::qk_fwd_kernel<decltype(d)::value><<<static_cast<unsigned>(blocks), 32 * qk::NW, 0, s>>>(p, per);
        return cudaGetLastError();
    });
}

cudaError_t launch_qk_bwd(const QkParams &p, cudaStream_t s) {
    const int32_t heads = p.Hq + p.Hk;
    const int per = qk::warps_per_token(p.rows, heads, p.D);
    const int32_t blocks = qk_bwd_blocks(p.rows, heads, p.D);
    const bool want = p.dq_weight || p.dk_weight;
    QkParams q = p;
    if (!want) q.partial = nullptr;
    cudaError_t err = qk::by_dim(p.D, [&](auto d) {
        constexpr int D = decltype(d)::value;
        if (p.dout_fp32)
            qk::qk_bwd_kernel<D, float><<<blocks, 32 * qk::NW, 0, s>>>(q, per, p.rows * per);
        else
            qk::qk_bwd_kernel<D, __nv_bfloat16><<<blocks, 32 * qk::NW, 0, s>>>(q, per, p.rows * per);
        return cudaGetLastError();
    });
    if (err != cudaSuccess || !want) return err;
    qk::qk_reduce_kernel<<<2 * p.D / 32, 256, 0, s>>>(q, blocks);
    return cudaGetLastError();
}

}  // namespace kda
