// kda_qk.cu -- per-head norm of queries and keys and their position rotation in one pass, and its gradient. sm_100a.
//
// For each token and head, with x the head's D channels:
//
//   r = (sum x^2 + eps)^(-1/2) (L2), (mean x^2 + eps)^(-1/2) (RMS) or 1;   z = x r w
//   (z_i, z_j) -> (z_i cos - z_j sin, z_j cos + z_i sin) for the pairs of the first `rot` channels,
//
// pairs (2i, 2i + 1) or (i, i + rot / 2), angle position * inv_freq_i, cos and sin times `factor`.
//
// Bound by HBM: 4 bytes per channel against some 20 operations, and nearly as much by the issue of those. D / 8
// lanes hold a head, so a warp takes 256 / D heads at a time. A lane has four pairs of channels, both channels
// of each, whatever the layout: 8 channels side by side (interleaved pairs, and channels that are not rotated),
// or 4 and the 4 that lie rot / 2 behind them. So the rotation needs no other lane, and arithmetic goes by
// packed pairs of fp32. Only the norm's sum crosses lanes.
//
// A warp walks the heads of a token, then those of its next token; its lanes' angles serve all heads of a token.
// Few tokens: several warps share one. The next heads arrive by asynchronous copies into a ring in shared
// memory, of which each thread reads back what it copied itself. (Shuffles for the half layout's partners, single
// fp32 operations: 179 instructions per pass and 84 us at 16384 x 40 heads x 128, where this takes 73.)
//
// An angle can be 10^6 radians, where 32 bits are off by 0.06. A lane keeps its frequencies as fractions of a turn
// in 64-bit fixed point; position times that, modulo 2^64, is the fraction of a turn to 2^-24 at worst (2^31
// tokens), and exact integer arithmetic (the same product in fp64 took longer than all the rest).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_qk.h"
#include "kda_seq.cuh"

namespace kda {
namespace qk {

constexpr int V = 8;              // channels per lane
constexpr int NW = 4;             // warps per CTA
constexpr int U = 2;              // passes computed side by side: a pass alone waits for its own sums
constexpr int kRing = 4;          // U passes each, whose loads are in flight: forward
constexpr int kBwdRing = 2;       // and backward, of q or k and of the gradient

// A lane's 8 channels as four pairs (a_i, b_i): a[0] = (a_0, a_1), a[1] = (a_2, a_3), and b.
struct Pairs {
    float2 a[2], b[2];
};
// where they are in the head: channels at[0] .. + 3 and at[1] .. + 3
struct Place {
    int at[2];
    bool turned, woven;   // rotated at all; (a_i, b_i) side by side
};
__device__ __forceinline__ Place place_of(const QkParams &p, int l) {
    Place q;
    q.turned = 8 * l < p.rot;
    q.woven = p.interleaved != 0;
    const bool apart = q.turned && !q.woven;
    q.at[0] = apart ? 4 * l : 8 * l;
    q.at[1] = apart ? 4 * l + (p.rot >> 1) : 8 * l + 4;
    return q;
}
__device__ __forceinline__ Pairs arrange(bool woven, const float (&x)[V]) {
    Pairs z;
    if (woven) {
        z.a[0] = make_float2(x[0], x[2]);
        z.a[1] = make_float2(x[4], x[6]);
        z.b[0] = make_float2(x[1], x[3]);
        z.b[1] = make_float2(x[5], x[7]);
    } else {
        z.a[0] = make_float2(x[0], x[1]);
        z.a[1] = make_float2(x[2], x[3]);
        z.b[0] = make_float2(x[4], x[5]);
        z.b[1] = make_float2(x[6], x[7]);
    }
    return z;
}
// `woven` is the same for all lanes
__device__ __forceinline__ Pairs from_bf16(bool woven, uint2 u, uint2 v) {
    const float x[V] = {bf_low(u.x), bf_high(u.x), bf_low(u.y), bf_high(u.y),
                        bf_low(v.x), bf_high(v.x), bf_low(v.y), bf_high(v.y)};
    return arrange(woven, x);
}
__device__ __forceinline__ void to_bf16(bool woven, const Pairs &z, uint16_t *head, const Place &q) {
    uint2 u, v;
    if (woven) {
        u = make_uint2(bf_pair(z.a[0].x, z.b[0].x), bf_pair(z.a[0].y, z.b[0].y));
        v = make_uint2(bf_pair(z.a[1].x, z.b[1].x), bf_pair(z.a[1].y, z.b[1].y));
    } else {
        u = make_uint2(bf_pair(z.a[0].x, z.a[0].y), bf_pair(z.a[1].x, z.a[1].y));
        v = make_uint2(bf_pair(z.b[0].x, z.b[0].y), bf_pair(z.b[1].x, z.b[1].y));
    }
    *reinterpret_cast<uint2 *>(head + q.at[0]) = u;
    *reinterpret_cast<uint2 *>(head + q.at[1]) = v;
}
__device__ __forceinline__ Pairs weights(const float *w, const Place &q) {
    float x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = w ? w[q.at[j >> 2] + (j & 3)] : 1.f;
    return arrange(q.woven, x);
}

// the lane's four angles, as frequencies in 2^-64 turns
struct Freq {
    uint64_t f[4];
};
// in the place of a frequency that is not finite: the 53 bits of an fp64 fraction of a turn leave the low bits of one
// from a half on 0, so no finite frequency has this value
constexpr uint64_t kNoFreq = (uint64_t(1) << 63) | 1;
__device__ __forceinline__ void make_freq(const QkParams &p, int l, const Place &q, Freq &r) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r.f[j] = 0;
        if (q.turned) {
            const double turns = static_cast<double>(p.inv_freq[4 * l + j]) * 0.15915494309189533577;
            r.f[j] = isfinite(turns) ? __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0) : kNoFreq;
        }
    }
}
// their cos and sin at a token, times the factor; sign: 1 forward, -1 for the transposed rotation
struct Turn {
    float2 c[2], s[2];
};
__device__ __forceinline__ void make_turn(const QkParams &p, int64_t row, const Place &q, float sign, const Freq &r, Turn &t) {
    float c[4], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        c[j] = 1.f;
        s[j] = 0.f;
    }
    if (q.turned) {
        const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(p.positions[row]));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // the top 32 bits as a signed fraction: -1/2 to 1/2 turn
            const int32_t top = static_cast<int32_t>((pos * r.f[j]) >> 32);
            sincospif(static_cast<float>(top) * 0x1p-31f, &s[j], &c[j]);
            c[j] *= p.factor;
            s[j] *= sign * p.factor;
            if (r.f[j] == kNoFreq) c[j] = s[j] = __int_as_float(0x7fffffff);   // a NaN at every position
        }
    }
    t.c[0] = make_float2(c[0], c[1]);
    t.c[1] = make_float2(c[2], c[3]);
    t.s[0] = make_float2(s[0], s[1]);
    t.s[1] = make_float2(s[2], s[3]);
}
__device__ __forceinline__ void rotate(const Turn &t, Pairs &z) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = z.a[i], b = z.b[i], minus = make_float2(-t.s[i].x, -t.s[i].y);
        z.a[i] = fma2(b, minus, mul2(a, t.c[i]));
        z.b[i] = fma2(a, t.s[i], mul2(b, t.c[i]));
    }
}
__device__ __forceinline__ float dot(const Pairs &x, const Pairs &y) {
    const float2 s = fma2(x.a[0], y.a[0], fma2(x.b[0], y.b[0], fma2(x.a[1], y.a[1], mul2(x.b[1], y.b[1]))));
    return s.x + s.y;
}
__device__ __forceinline__ void times(Pairs &z, const Pairs &w) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        z.a[i] = mul2(z.a[i], w.a[i]);
        z.b[i] = mul2(z.b[i], w.b[i]);
    }
}
__device__ __forceinline__ void times(Pairs &z, float f) {
    const float2 g = make_float2(f, f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        z.a[i] = mul2(z.a[i], g);
        z.b[i] = mul2(z.b[i], g);
    }
}
// z += x y
__device__ __forceinline__ void add_product(Pairs &z, const Pairs &x, const Pairs &y) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        z.a[i] = fma2(x.a[i], y.a[i], z.a[i]);
        z.b[i] = fma2(x.b[i], y.b[i], z.b[i]);
    }
}

template <int LPH>
__device__ __forceinline__ void head_sums(float (&x)[U]) {
#pragma unroll
    for (int d = LPH / 2; d > 0; d >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] += __shfl_xor_sync(0xffffffffu, x[u], d);
}

// 1 / norm of each pass's head; a zero vector without eps stays zero
template <int D>
__device__ __forceinline__ void inverse_norms(const QkParams &p, const Pairs (&x)[U], float (&r)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = 1.f;
    if (p.norm == kNormNone) return;   // the same for all lanes
    float ss[U];
#pragma unroll
    for (int u = 0; u < U; ++u) ss[u] = dot(x[u], x[u]);
    head_sums<D / V>(ss);
    const float share = p.norm == kNormRms ? 1.f / D : 1.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float t = fmaf(ss[u], share, p.eps);
        r[u] = t == 0.f ? 0.f : rsqrtf(t);
    }
}

// A warp's passes. A pass is 256 / D heads of q, or as many of k; task t is a token's passes, or with per_token > 1 every
// per_token-th of them; a warp takes task t, t + stride, ... The rows' places are kept as pointers, so that a
// step from pass to pass is a shift and an addition (with 64-bit products per pass it took as long as the rest).
struct Cursor {
    int64_t task, row;
    int pass;
};
__device__ __forceinline__ void start(Cursor &c, int64_t task, int per_token) {
    c.task = task;
    c.row = task / per_token;
    c.pass = static_cast<int>(task - c.row * per_token);
}
// U passes on; whether those are another token's
__device__ __forceinline__ bool advance(Cursor &c, int per_token, int passes, int64_t stride) {
    c.pass += U * per_token;
    if (c.pass < passes) return false;
    start(c, c.task + stride, per_token);
    return true;
}

template <int kBytes>
__device__ __forceinline__ void copy(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "n"(kBytes)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <int D>
__global__ void __launch_bounds__(32 * NW) qk_fwd_kernel(QkParams p, int per_token, int64_t tasks) {
    constexpr int LPH = D / V, HPW = 32 / LPH, PW = HPW * D;   // PW: channels per pass
    __shared__ __align__(16) uint2 ring[NW][kRing][U][2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH;
    const int pq = (p.Hq + HPW - 1) / HPW, passes = pq + (p.Hk + HPW - 1) / HPW;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * NW;
    const bool woven = p.interleaved != 0;
    const Place place = place_of(p, l);
    uint2(*mine)[U][2][32] = ring[warp];
    Cursor at = {}, ahead = {};
    start(at, static_cast<int64_t>(blockIdx.x) * NW + warp, per_token);
    ahead = at;
    const uint16_t *qi = p.q + ahead.row * p.q_stride + sub * D, *ki = p.k + ahead.row * p.k_stride + sub * D;
    int put = 0;
    auto fetch = [&]() {
        if (ahead.task < tasks) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int pass = ahead.pass + u * per_token;
                const bool is_q = pass < pq;
                const int n = is_q ? pass : pass - pq;
                if (n * HPW + sub < (is_q ? p.Hq : p.Hk)) {
                    const uint16_t *head = (is_q ? qi : ki) + n * PW;
                    copy<8>(&mine[put][u][0][lane], head + place.at[0]);
                    copy<8>(&mine[put][u][1][lane], head + place.at[1]);
                }
            }
            if (advance(ahead, per_token, passes, stride)) {
                qi = p.q + ahead.row * p.q_stride + sub * D;
                ki = p.k + ahead.row * p.k_stride + sub * D;
            }
        }
        put = (put + 1) & (kRing - 1);
        copy_commit();
    };
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) fetch();
    Turn t;
    Freq f;
    make_freq(p, l, place, f);
    const Pairs wq = weights(p.q_weight, place), wk = weights(p.k_weight, place);
    bool fresh = true;
    uint16_t *qo = nullptr, *ko = nullptr;
    for (int get = 0; at.task < tasks; get = (get + 1) & (kRing - 1)) {
        fetch();
        if (fresh) {
            make_turn(p, at.row, place, 1.f, f, t);
            qo = p.q_out + at.row * p.q_out_stride + sub * D;
            ko = p.k_out + at.row * p.k_out_stride + sub * D;
        }
        copy_wait<kRing - 1>();
        Pairs z[U];
        float r[U];
        bool is_q[U], there[U];
        int n[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int pass = at.pass + u * per_token;
            is_q[u] = pass < pq;
            n[u] = is_q[u] ? pass : pass - pq;
            there[u] = n[u] * HPW + sub < (is_q[u] ? p.Hq : p.Hk);
            // where there is no head: what an earlier pass left there, and nothing comes of it
            z[u] = from_bf16(woven, mine[get][u][0][lane], mine[get][u][1][lane]);
        }
        inverse_norms<D>(p, z, r);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (is_q[u] ? p.q_weight != nullptr : p.k_weight != nullptr) times(z[u], is_q[u] ? wq : wk);
            if (p.norm != kNormNone) times(z[u], r[u]);
            if (p.rot) rotate(t, z[u]);
            if (there[u]) to_bf16(woven, z[u], (is_q[u] ? qo : ko) + n[u] * PW, place);
        }
        fresh = advance(at, per_token, passes, stride);
    }
}

// Gradients: dz is the rotation's transpose applied to the given gradient,
//   dx = r (w dz - xh <xh, w dz> / (1 or D)),  xh = x r,   dw = sum over tokens and heads of dz xh.
// CTAs walk the tasks, so that there are few partial sums of dw; they are added in a fixed order. (2 x 4096 x 64 heads
// x 128, bf16: 91 us, and 6 for the sums; 4.4 TB/s. The issue of its 30 operations per channel is as near a bound.)
template <int D, class TD>
__global__ void __launch_bounds__(32 * NW) qk_bwd_kernel(QkParams p, int per_token, int64_t tasks) {
    constexpr int LPH = D / V, HPW = 32 / LPH, PW = HPW * D;
    constexpr int kG = 4 * sizeof(TD);                          // bytes of four channels' gradient
    constexpr int kPass = 2 * 32 * (8 + kG);                    // a pass in the ring: [2][32] of x, then of the gradient
    constexpr int kRingBytes = NW * kBwdRing * U * kPass, kPartBytes = NW * HPW * D * 4;
    __shared__ __align__(16) uint8_t shared[kRingBytes > kPartBytes ? kRingBytes : kPartBytes];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH;
    const int pq = (p.Hq + HPW - 1) / HPW, passes = pq + (p.Hk + HPW - 1) / HPW;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * NW;
    const bool woven = p.interleaved != 0;
    const Place place = place_of(p, l);
    uint8_t *mine = shared + warp * kBwdRing * U * kPass;
    Cursor at = {}, ahead = {};
    start(at, static_cast<int64_t>(blockIdx.x) * NW + warp, per_token);
    ahead = at;
    const uint16_t *qi, *ki;
    const TD *dqi, *dki;
    auto rows = [&]() {
        qi = p.q + ahead.row * p.q_stride + sub * D;
        ki = p.k + ahead.row * p.k_stride + sub * D;
        dqi = static_cast<const TD *>(p.dq_out) + ahead.row * p.dq_stride + sub * D;
        dki = static_cast<const TD *>(p.dk_out) + ahead.row * p.dk_stride + sub * D;
    };
    rows();
    int put = 0;
    auto fetch = [&]() {
        if (ahead.task < tasks) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int pass = ahead.pass + u * per_token;
                const bool is_q = pass < pq;
                const int n = is_q ? pass : pass - pq;
                if (n * HPW + sub < (is_q ? p.Hq : p.Hk)) {
                    uint8_t *to = mine + (put * U + u) * kPass;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        copy<8>(to + (32 * i + lane) * 8, (is_q ? qi : ki) + n * PW + place.at[i]);
                        copy<kG>(to + 512 + (32 * i + lane) * kG, (is_q ? dqi : dki) + n * PW + place.at[i]);
                    }
                }
            }
            if (advance(ahead, per_token, passes, stride)) rows();
        }
        put = (put + 1) & (kBwdRing - 1);
        copy_commit();
    };
#pragma unroll
    for (int k = 0; k < kBwdRing - 1; ++k) fetch();
    Turn t;
    Freq f;
    make_freq(p, l, place, f);
    const Pairs wq = weights(p.q_weight, place), wk = weights(p.k_weight, place);
    Pairs dwq, dwk;
#pragma unroll
    for (int i = 0; i < 2; ++i) dwq.a[i] = dwq.b[i] = dwk.a[i] = dwk.b[i] = make_float2(0.f, 0.f);
    const float share = p.norm == kNormRms ? 1.f / D : 1.f;
    bool fresh = true;
    uint16_t *qo = nullptr, *ko = nullptr;
    for (int get = 0; at.task < tasks; get = (get + 1) & (kBwdRing - 1)) {
        fetch();
        if (fresh) {
            make_turn(p, at.row, place, -1.f, f, t);
            qo = p.q_out + at.row * p.q_out_stride + sub * D;
            ko = p.k_out + at.row * p.k_out_stride + sub * D;
        }
        copy_wait<kBwdRing - 1>();
        Pairs x[U], d[U];
        float r[U], along[U];
        bool is_q[U], there[U];
        int n[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int pass = at.pass + u * per_token;
            is_q[u] = pass < pq;
            n[u] = is_q[u] ? pass : pass - pq;
            there[u] = n[u] * HPW + sub < (is_q[u] ? p.Hq : p.Hk);
            const uint8_t *from = mine + (get * U + u) * kPass;
            const uint2 *fx = reinterpret_cast<const uint2 *>(from) + lane;
            // where there is no head, zeros: they enter the weights' sums
            const uint2 none = make_uint2(0u, 0u);
            x[u] = from_bf16(woven, there[u] ? fx[0] : none, there[u] ? fx[32] : none);
            if constexpr (sizeof(TD) == 2) {
                const uint2 *fd = reinterpret_cast<const uint2 *>(from + 512) + lane;
                d[u] = from_bf16(woven, there[u] ? fd[0] : none, there[u] ? fd[32] : none);
            } else {
                const float4 *fd = reinterpret_cast<const float4 *>(from + 512) + lane, zero = make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 g = there[u] ? fd[0] : zero, h = there[u] ? fd[32] : zero;
                const float y[V] = {g.x, g.y, g.z, g.w, h.x, h.y, h.z, h.w};
                d[u] = arrange(woven, y);
            }
            if (p.rot) rotate(t, d[u]);
        }
        inverse_norms<D>(p, x, r);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            times(x[u], r[u]);
            if (is_q[u]) {
                add_product(dwq, d[u], x[u]);
                times(d[u], wq);
            } else {
                add_product(dwk, d[u], x[u]);
                times(d[u], wk);
            }
            along[u] = dot(d[u], x[u]);
        }
        if (p.norm != kNormNone) {
            head_sums<LPH>(along);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float m = -along[u] * share;
                Pairs back;
#pragma unroll
                for (int i = 0; i < 2; ++i) back.a[i] = back.b[i] = make_float2(m, m);
                add_product(d[u], x[u], back);
                times(d[u], r[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (there[u]) to_bf16(woven, d[u], (is_q[u] ? qo : ko) + n[u] * PW, place);
        fresh = advance(at, per_token, passes, stride);
    }
    if (!p.partial) return;
    copy_wait<0>();
    float(*part)[HPW][D] = reinterpret_cast<float(*)[HPW][D]>(shared);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) {
            // channel j of the lane: its place among the pairs
            const Pairs &dw = which ? dwk : dwq;
            const int i = woven ? j >> 1 : j & 3;
            const float2 of = (woven ? j & 1 : j >> 2) ? dw.b[i >> 1] : dw.a[i >> 1];
            part[warp][sub][place.at[j >> 2] + (j & 3)] = i & 1 ? of.y : of.x;
        }
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

// grid 2 D / 32: 32 sums per CTA, 32 threads each
__global__ void __launch_bounds__(1024) qk_reduce_kernel(QkParams p, int blocks) {
    __shared__ float part[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, at = blockIdx.x * 32 + x;
    float s = 0.f;
#pragma unroll 4
    for (int b = y; b < blocks; b += 32) s += p.partial[static_cast<int64_t>(b) * 2 * p.D + at];
    part[y][x] = s;
    __syncthreads();
    // warp y adds up column y
    s = part[x][y];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (x == 0) {
        const int c = blockIdx.x * 32 + y;
        if (c < p.D) {
            if (p.dq_weight) p.dq_weight[c] = s;
        } else if (p.dk_weight) {
            p.dk_weight[c - p.D] = s;
        }
    }
}

// warps per token: one where that makes 16 warps per SM, else as many as it takes, up to one per pass
int warps_per_token(int64_t rows, int32_t heads, int32_t D) {
    const int passes = (heads * D + 255) / 256;   // or one more, where q or k do not fill their last
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

// CTAs that walk the tasks: at most `most` per SM, and no more than it takes for all warps to have equally many
int32_t walkers(int64_t tasks, int most) {
    const int64_t n = (tasks + qk::NW - 1) / qk::NW, each = (n + most * 148 - 1) / (most * 148);
    return n < 1 ? 1 : static_cast<int32_t>((n + each - 1) / each);
}

int32_t qk_bwd_blocks(int64_t rows, int32_t heads, int32_t D) {
    return walkers(rows * qk::warps_per_token(rows, heads, D), 8);
}

cudaError_t launch_qk_fwd(const QkParams &p, cudaStream_t s) {
    if (p.rows == 0) return cudaSuccess;
    const int per = qk::warps_per_token(p.rows, p.Hq + p.Hk, p.D);
    const int32_t blocks = walkers(p.rows * per, 16);
    return qk::by_dim(p.D, [&](auto d) {
        qk::qk_fwd_kernel<decltype(d)::value><<<blocks, 32 * qk::NW, 0, s>>>(p, per, p.rows * per);
        return cudaGetLastError();
    });
}

cudaError_t launch_qk_bwd(const QkParams &p, cudaStream_t s) {
    if (p.rows == 0) {
        // no token, so the weights' gradients are zero; the other inputs may be NULL, and no kernel reads them
        cudaError_t err = cudaSuccess;
        for (float *dw : {p.dq_weight, p.dk_weight})
            if (dw && err == cudaSuccess) err = cudaMemsetAsync(dw, 0, p.D * sizeof(float), s);
        return err;
    }
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
    qk::qk_reduce_kernel<<<2 * p.D / 32, 1024, 0, s>>>(q, blocks);
    return cudaGetLastError();
}

}  // namespace kda
