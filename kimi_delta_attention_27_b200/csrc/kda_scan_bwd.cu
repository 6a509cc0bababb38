// kda_scan_bwd.cu -- gradients of the selective state space scan, sm_100a.
//
// With the forward's tile (64 tokens, entering state S_0, Gamma, L; see kda_scan_fwd.cu) and R the gradient of
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
// is taken elementwise in fp32; dy S_0^T and x R^T, from which fp32 results follow, take S_0 and R as three
// bf16 parts (24 bits). M, K and the copy of R that makes dx are rounded to bf16 once, for results in bf16.
//
// The states S_0 and gradients R of every tile come from two sweeps (launch_scan_states), fp32 in the
// workspace. The gradient kernel then takes all tiles at once: the one of this file at a state size of 64, that of
// kda_scan_tc_bwd.cu, with tiles of 128 tokens, at 128. Here one CTA has one tile of one group and walks (a share of)
// the group's heads, so C B^T is computed once, and dB and dC add up over the heads in registers, without atomics:
// N / 16 warps own 16 columns of dC each and multiply with S_0, N / 16 others own dB and multiply with R; Q, M, K and
// dx are shared out over all of them. The next head's x and dy, and once this one's have been used its S_0 and R, arrive
// by TMA. Where tiles x groups leave SMs idle the heads are shared out over several CTAs, whose dB and dC are added by
// scan_bc_kernel in a fixed order. Sums over tokens go by partial sums per tile, too: runs repeat bit for bit.
//
// Bound by shared memory, which the fragments of every product come from, and by the chain of a head's phases: 5 packed
// sequences, 5001 tokens x 32 heads x 128, 2 groups, 64 entries: 192 us (198 with a head's steps waited for at the head;
// the workspace's 0.33 GB alone is 50 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_scan_tc.cuh"

namespace kda {
namespace scan {

struct BwdGates : Gates {
    float slope[T];   // of the step in dt
    float A, D, pad2[2];
};

constexpr int N = 64;

struct BwdSmem {
    static constexpr int NW = N / 16;                      // warps for dC, and as many for dB: 16 columns each
    static constexpr int kBC = T * N * 2, kX = T * PC * 2, kM = T * T * 2;
    static constexpr int kB = 0, kC = kBC;
    static constexpr int kXY = 2 * kBC;                    // two stages of x and dy
    static constexpr int kMt = kXY + 4 * kX, kKt = kMt + kM;
    static constexpr int kR = kKt + kM;                    // R in bf16, N x 64
    static constexpr int kGates = kR + N * PC * 2;
    static constexpr int kRow = kGates + 3 * static_cast<int>(sizeof(BwdGates));   // [8][T] row sums of M . Q d
    static constexpr int kCol = kRow + 8 * T * 4;          // [4][T] column sums of M . Q, without the diagonal
    static constexpr int kDiag = kCol + 4 * T * 4;         // [2][T] the diagonals of M . Q and of Q
    static constexpr int kInt = kDiag + 2 * T * 4;         // [2][NW][T] C . (S_0 dy) and B . (R x)
    static constexpr int kRS = kInt + 2 * NW * T * 4;      // [2 NW] <R, S_0>
    static constexpr int kTok = kRS + 64;                  // [5][T] per token, summed over a head's slices; <R, S_0>
    static constexpr int kNext = kTok + 5 * T * 4 + 16;    // the next head's dt, A, bias and D
    static constexpr int kBars = kNext + (T + 4) * 4;
    static constexpr int kState = (kBars + 64 + 1023) / 1024 * 1024;   // S_0, R: each two blocks of 32 columns
    static constexpr int kBytes = kState + 2 * N * PC * 4;
    static_assert(kBytes + 1024 <= 227 * 1024, "shared memory of one CTA");
};

// 16 x 8 blocks of the lower triangle of a 64 x 64 matrix: row block 0 has 2, 1 has 4, 2 has 6, 3 has 8
__device__ __forceinline__ void triangle_block(int j, int &rb, int &cb) {
    rb = j < 2 ? 0 : j < 6 ? 1 : j < 12 ? 2 : 3;
    cb = j - rb * (rb + 1);
}

__device__ unsigned int g_scan_bwd_error = 0;

struct BwdMaps {
    CUtensorMap x, dy, states, grads;
};

// two consecutive columns of two rows of a state as a B fragment in S parts: element [n][p], k = p
template <int S>
__device__ __forceinline__ void state_frag(const float2 &v0, const float2 &v1, uint32_t (&b)[S][2]) {
    uint32_t part[S];
    split<S>(v0.x, v0.y, part);
#pragma unroll
    for (int s = 0; s < S; ++s) b[s][0] = part[s];
    split<S>(v1.x, v1.y, part);
#pragma unroll
    for (int s = 0; s < S; ++s) b[s][1] = part[s];
}

__global__ void __launch_bounds__(4 * N, 1) scan_bwd_kernel(ScanParams p, BwdWork w, const __grid_constant__ BwdMaps maps) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = BwdSmem;
    constexpr int NW = L::NW, ALL = 2 * NW, NT = 32 * ALL, ROWB = N * 2, BLOCKS = (20 + ALL - 1) / ALL, XT = 32 / ALL;
    const uint32_t base = smem_addr(smem);
    BwdGates *gates = reinterpret_cast<BwdGates *>(smem + L::kGates);
    float *rows_s = reinterpret_cast<float *>(smem + L::kRow), *cols_s = reinterpret_cast<float *>(smem + L::kCol);
    float *diag_s = reinterpret_cast<float *>(smem + L::kDiag), *int_s = reinterpret_cast<float *>(smem + L::kInt);
    float *rs_s = reinterpret_cast<float *>(smem + L::kRS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gl = lane >> 2, q2 = (lane & 3) * 2;
    const int which = warp / NW, cw = warp % NW;   // 0: dC and S_0, 1: dB and R; columns 16 cw .. + 16
    const int split_i = static_cast<int>(blockIdx.x % w.splits);
    const int grp = static_cast<int>(blockIdx.x / w.splits % p.G);
    const int64_t unit = blockIdx.x / w.splits / p.G;
    const int per_group = p.H / p.G, per = (per_group + w.splits - 1) / w.splits;
    const int hb = grp * per_group + split_i * per;
    const int he = min(hb + per, (grp + 1) * per_group);
    const Piece u = find_piece(p.seqs, unit, T);
    const int cnt = u.none ? 0 : static_cast<int>(u.b - u.a);
    if (cnt == 0) {
        for (int j = tid; j < 3 * (he - hb); j += NT)
            w.part[(unit * 3 + j / (he - hb)) * p.H + hb + j % (he - hb)] = 0.f;
        return;
    }
    const int slices = p.P / PC, work = (he - hb) * slices;
    if (work <= 0) return;
    const int64_t start = u.a;

    __shared__ uint32_t s_abort;
    tc::Ctx x;
    x.bars = base + L::kBars;   // 0, 1: x and dy of a stage; 2: S_0 and R
    x.abort = &s_abort;
    x.error = &g_scan_bwd_error;
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) ptx::mbar_init(x.bar(i), 1);
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    // Gates, by one warp: what they take from memory is on its way a head ahead.
    // Lane l copies and reads tokens 2l and 2l + 1; the last three words go through a lane each.
    const float *next_s = reinterpret_cast<const float *>(smem + L::kNext);
    auto fetch_gates = [&](int h) {
        const uint32_t d = base + L::kNext;
        const float *src = p.dt + start * p.H + h;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            cp_async4(d + t * 4, src + (t < cnt ? static_cast<int64_t>(t) * p.H : 0), t < cnt);
        }
        if (lane < 3) {
            const float *f = lane == 0 ? p.A : lane == 1 ? p.dt_bias : p.D;
            cp_async4(d + (T + lane) * 4, (f ? f : p.A) + h, f != nullptr);
        }
        cp_async_commit();
    };
    auto make_head = [&](BwdGates &g) {
        cp_async_wait_all();
        __syncwarp();
        const float A = next_s[T], bias = next_s[T + 1];
        float d[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            float u;
            d[e] = step_of(next_s[t], bias, p.softplus, &u);
            if (t >= cnt) d[e] = 0.f;
            g.slope[t] = p.softplus ? 1.f / (1.f + expf(-u)) : 1.f;
        }
        make_gates(g, d[0], d[1], A);
        if (lane == 0) {
            g.A = A;
            g.D = next_s[T + 2];
        }
        __syncwarp();
    };
    // by one thread
    auto fetch = [&](int k, int stage) {
        const int32_t col = (hb + k / slices) * p.P + (k % slices) * PC, row = static_cast<int32_t>(start);
        const uint32_t d = base + L::kXY + stage * 2 * L::kX;
        ptx::mbar_arrive_expect_tx(x.bar(stage), 2 * L::kX);
        tc::tma_load_2d(d, &maps.x, x.bar(stage), col, row);
        tc::tma_load_2d(d + L::kX, &maps.dy, x.bar(stage), col, row);
    };
    auto fetch_state = [&](int k) {
        const int32_t row = static_cast<int32_t>((unit * p.H + hb + k / slices) * N), col = (k % slices) * PC;
        ptx::mbar_arrive_expect_tx(x.bar(2), 2 * N * PC * 4);
        for (int j = 0; j < 2; ++j) {
            tc::tma_load_2d(base + L::kState + j * N * 128, &maps.states, x.bar(2), col + 32 * j, row);
            tc::tma_load_2d(base + L::kState + (2 + j) * N * 128, &maps.grads, x.bar(2), col + 32 * j, row);
        }
    };
    load_tile<ROWB, NT>(base + L::kB, p.B + start * p.b_stride + static_cast<int64_t>(grp) * N, p.b_stride, cnt);
    load_tile<ROWB, NT>(base + L::kC, p.C + start * p.c_stride + static_cast<int64_t>(grp) * N, p.c_stride, cnt);
    cp_async_commit();
    if (tid == 0) {
        fetch(0, 0);
        fetch_state(0);
    }
    if (warp == NW - 2) {
        fetch_gates(hb);
        make_head(gates[0]);
        if (hb + 1 < he) fetch_gates(hb + 1);
    }
    cp_async_wait_all();
    __syncthreads();

    // C B^T, the blocks of the lower triangle that this warp keeps
    float cb_acc[BLOCKS][4];
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j) {
        cb_acc[j][0] = cb_acc[j][1] = cb_acc[j][2] = cb_acc[j][3] = 0.f;
        if (warp + j * ALL < 20) {
            int rb, cb;
            triangle_block(warp + j * ALL, rb, cb);
#pragma unroll
            for (int k = 0; k < N / 16; ++k) {
                uint32_t a[4], b[4];
                frag_a<ROWB>(base + L::kC, rb * 16, 2 * k, a);
                frag_b<ROWB>(base + L::kB, (cb >> 1) * 16, 2 * k, b);
                mma(cb_acc[j], a, cb & 1 ? b[2] : b[0], cb & 1 ? b[3] : b[1]);
            }
        }
    }
    float acc[4][2][4];   // dC or dB: rows 16 m, columns 16 cw + 8 n
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
    // this warp's rows of S_0 (of 0) or R (1) as B fragments: row 8 n + gl, columns 16 kk + q2 + 8 x, + 1
    auto state_at = [&](int of, int kk, int n, int x8) {
        const int row = cw * 16 + 8 * n + gl, chunk = (kk & 1) * 4 + 2 * x8 + (q2 >> 2);
        return *reinterpret_cast<const float2 *>(smem + L::kState + (2 * of + (kk >> 1)) * N * 128 + at<128>(row, chunk) +
                                                 (q2 & 3) * 4);
    };
    float *tok_s = reinterpret_cast<float *>(smem + L::kTok);   // q, int, in, dd, Q_tt (see below)

    // The steps' gradients of head h from its tokens' sums, by one warp (lane l: tokens 2l and 2l + 1).
    auto finish_head = [&](int h, const BwdGates &g) {
        float v[10];
#pragma unroll
        for (int j = 0; j < 5; ++j) {
            const float2 f = reinterpret_cast<const float2 *>(tok_s + j * T)[lane];
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
        // suffix sums of q + int, prefix sums of in
        float suf = v[0] + v[2] + v[1] + v[3], pre = v[4] + v[5];
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const float a = __shfl_down_sync(0xffffffffu, suf, x), b = __shfl_up_sync(0xffffffffu, pre, x);
            if (lane + x < 32) suf += a;
            if (lane >= x) pre += b;
        }
        // behind the lane's tokens, and before them
        float after = __shfl_down_sync(0xffffffffu, suf, 1), before = __shfl_up_sync(0xffffffffu, pre, 1);
        if (lane == 31) after = 0.f;
        if (lane == 0) before = 0.f;
        const float rest = g.total * tok_s[5 * T];
        const float dl[2] = {suf + (before + rest), after + (v[1] + v[3]) + (before + v[4] + rest)};
        float sa = 0.f, sb = 0.f, sd = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            if (t < cnt) {
                const float dd = fmaf(dl[e], g.A, v[6 + e]) * g.slope[t];
                p.ddt[(start + t) * p.H + h] = dd;
                sa = fmaf(dl[e], g.d[t], sa);
                sb += dd;
                sd += v[8 + e];
            }
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) {
            sa += __shfl_xor_sync(0xffffffffu, sa, x);
            sb += __shfl_xor_sync(0xffffffffu, sb, x);
            sd += __shfl_xor_sync(0xffffffffu, sd, x);
        }
        if (lane == 0) {
            w.part[(unit * 3 + 0) * p.H + h] = sa;
            w.part[(unit * 3 + 1) * p.H + h] = sb;
            w.part[(unit * 3 + 2) * p.H + h] = sd;
        }
    };

    bool ok = true;
    for (int k = 0; k < work; ++k) {
        const int h = hb + k / slices, sl = k % slices, stage = k & 1;
        const BwdGates &g = gates[(k / slices) % 3];
        const uint32_t xt = base + L::kXY + stage * 2 * L::kX, dyt = xt + L::kX;
        // all of the last head's sums, M, K and the other stage are free
        if (k > 0 && __syncthreads_or(!ok)) break;
        if (tid == 0 && k + 1 < work) fetch(k + 1, stage ^ 1);
        ok &= x.wait(stage, (k >> 1) & 1);
        if (cnt < T) {
            // rows behind the piece: of other tokens, or none
            for (int j = tid; j < (T - cnt) * 16; j += NT) {
                const int r = cnt + (j >> 4), c = j & 15;
                *reinterpret_cast<uint4 *>(smem + (xt - base) + (c >> 3) * L::kX + r * 128 + (c & 7) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            ptx::fence_proxy_async_smem();
            __syncthreads();
        }
        // ---- Q, M, K and the sums of M . Q; the blocks' products side by side
        float qs[BLOCKS][4];
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j) qs[j][0] = qs[j][1] = qs[j][2] = qs[j][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < PC / 16; ++kk) {
            uint32_t a[BLOCKS][4], b[BLOCKS][4];
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j) {
                if (warp + j * ALL < 20) {
                    int rb, cb;
                    triangle_block(warp + j * ALL, rb, cb);
                    frag_a<PC * 2>(dyt, rb * 16, 2 * kk, a[j]);
                    frag_b<PC * 2>(xt, (cb >> 1) * 16, 2 * kk, b[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j) {
                if (warp + j * ALL < 20) {
                    int rb, cb;
                    triangle_block(warp + j * ALL, rb, cb);
                    mma(qs[j], a[j], cb & 1 ? b[j][2] : b[j][0], cb & 1 ? b[j][3] : b[j][1]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j) {
            if (warp + j * ALL < 20) {
                int rb, cb;
                triangle_block(warp + j * ALL, rb, cb);
                const float(&qa)[4] = qs[j];
                const int r = rb * 16 + gl, s = cb * 8 + q2;
                float rsum[2] = {0.f, 0.f}, csum[2] = {0.f, 0.f}, mv[4], kv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = r + (e >> 1) * 8, c = s + (e & 1);
                    const float l = c <= t ? ex2((g.hi[t] - g.hi[c]) + (g.lo[t] - g.lo[c])) : 0.f;
                    // selected, not multiplied: what lies above the diagonal may be anything
                    mv[e] = c <= t ? cb_acc[j][e] * l : 0.f;
                    const float ql = c <= t ? qa[e] * l : 0.f;
                    kv[e] = ql * g.d[c];
                    const float hq = c < t ? mv[e] * qa[e] : 0.f;
                    rsum[e >> 1] = fmaf(hq, g.d[c], rsum[e >> 1]);
                    csum[e & 1] += hq;
                    if (c == t) {
                        diag_s[t] = mv[e] * qa[e];
                        diag_s[T + t] = qa[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t off = at<T * 2>(r + 8 * e, cb) + q2 * 2;
                    *reinterpret_cast<uint32_t *>(smem + L::kMt + off) = bf_pair(mv[2 * e], mv[2 * e + 1]);
                    *reinterpret_cast<uint32_t *>(smem + L::kKt + off) = bf_pair(kv[2 * e], kv[2 * e + 1]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    rsum[e] += __shfl_xor_sync(0xffffffffu, rsum[e], 1);
                    rsum[e] += __shfl_xor_sync(0xffffffffu, rsum[e], 2);
                    csum[e] += __shfl_xor_sync(0xffffffffu, csum[e], 4);
                    csum[e] += __shfl_xor_sync(0xffffffffu, csum[e], 8);
                    csum[e] += __shfl_xor_sync(0xffffffffu, csum[e], 16);
                }
                if ((lane & 3) == 0) {
                    rows_s[cb * T + r] = rsum[0];
                    rows_s[cb * T + r + 8] = rsum[1];
                }
                if (gl == 0) {
                    cols_s[rb * T + s] = csum[0];
                    cols_s[rb * T + s + 1] = csum[1];
                }
            }
        }
        // ---- dy S_0^T or x R^T: 64 x 16 for this warp
        ok &= x.wait(2, k & 1);
        {
            const uint32_t at_tile = which ? xt : dyt, bc = which ? L::kB : L::kC;
            float tmp[4][2][4], rs = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n) tmp[m][n][0] = tmp[m][n][1] = tmp[m][n][2] = tmp[m][n][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t b[2][3][2];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 v0 = state_at(which, kk, n, 0), v1 = state_at(which, kk, n, 1);
                    state_frag<3>(v0, v1, b[n]);
                    if (which) {
                        const int row = cw * 16 + 8 * n + gl;
                        *reinterpret_cast<uint32_t *>(smem + L::kR + at<PC * 2>(row, 2 * kk) + q2 * 2) = b[n][0][0];
                        *reinterpret_cast<uint32_t *>(smem + L::kR + at<PC * 2>(row, 2 * kk + 1) + q2 * 2) = b[n][0][1];
                    }
                    if (which == (kk >> 1)) {
                        // <R, S_0>, half of the columns each
                        const float2 s0 = state_at(1 - which, kk, n, 0), s1 = state_at(1 - which, kk, n, 1);
                        rs = fmaf(s0.x, v0.x, fmaf(s0.y, v0.y, fmaf(s1.x, v1.x, fmaf(s1.y, v1.y, rs))));
                    }
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t a[4];
                    frag_a<PC * 2>(at_tile, m * 16, 2 * kk, a);
#pragma unroll
                    for (int s = 2; s >= 0; --s)
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma(tmp[m][n], a, b[n][s][0], b[n][s][1]);
                }
            }
            // the dot with C's or B's own columns, and into dC or dB
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = m * 16 + 8 * e + gl;
                    const float f = which ? g.weight[t] : g.from[t];
                    float dot = 0.f;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const uint32_t cv = *reinterpret_cast<const uint32_t *>(smem + bc + at<ROWB>(t, 2 * cw + n) + q2 * 2);
                        dot = fmaf(tmp[m][n][2 * e], bf_low(cv), fmaf(tmp[m][n][2 * e + 1], bf_high(cv), dot));
                        acc[m][n][2 * e] = fmaf(f, tmp[m][n][2 * e], acc[m][n][2 * e]);
                        acc[m][n][2 * e + 1] = fmaf(f, tmp[m][n][2 * e + 1], acc[m][n][2 * e + 1]);
                    }
                    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
                    dot += __shfl_xor_sync(0xffffffffu, dot, 2);
                    if ((lane & 3) == 0) int_s[(which * NW + cw) * T + t] = dot;
                }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, x);
            if (lane == 0) rs_s[warp] = rs;
        }
        // by warps with the fewest blocks above: the last head's steps, whose tokens' sums are complete, and the next
        // head's gates (its own buffer: the last one's are in use)
        if (warp == NW - 1 && sl == 0 && k > 0) finish_head(h - 1, gates[(k / slices + 2) % 3]);
        if (warp == NW - 2 && sl == slices - 1 && h + 1 < he) {
            make_head(gates[(k / slices + 1) % 3]);
            if (h + 2 < he) fetch_gates(h + 2);
        }
        __syncthreads();   // M, K, R and the sums are complete, S_0 and R used
        if (tid == 0 && k + 1 < work) {
            ptx::fence_proxy_async_smem();
            fetch_state(k + 1);
        }
        // ---- dC += K B, dB += K^T C
        if (which == 0) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t b[4];
                frag_bt<ROWB>(base + L::kB, kk * 16, 2 * cw, b);
#pragma unroll
                for (int m = kk; m < 4; ++m) {
                    uint32_t a[4];
                    frag_a<T * 2>(base + L::kKt, m * 16, 2 * kk, a);
                    mma(acc[m][0], a, b[0], b[1]);
                    mma(acc[m][1], a, b[2], b[3]);
                }
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t b[4];
                frag_bt<ROWB>(base + L::kC, kk * 16, 2 * cw, b);
#pragma unroll
                for (int m = 0; m <= kk; ++m) {
                    uint32_t a[4];
                    frag_at<T * 2>(base + L::kKt, kk * 16, 2 * m, a);
                    mma(acc[m][0], a, b[0], b[1]);
                    mma(acc[m][1], a, b[2], b[3]);
                }
            }
        }
        // ---- dx: rows 16 (warp % 4), XT 8-column tiles
        {
            const int r0 = (warp & 3) * 16, c0 = (warp >> 2) * XT, row = r0 + gl;
            float out[XT][4];
#pragma unroll
            for (int j = 0; j < XT; ++j) out[j][0] = out[j][1] = out[j][2] = out[j][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < N / 16; ++kk) {
                uint32_t a[4];
                frag_a<ROWB>(base + L::kB, r0, 2 * kk, a);
#pragma unroll
                for (int j = 0; j < XT / 2; ++j) {
                    uint32_t b[4];
                    frag_bt<PC * 2>(base + L::kR, kk * 16, c0 + 2 * j, b);
                    mma(out[2 * j], a, b[0], b[1]);
                    mma(out[2 * j + 1], a, b[2], b[3]);
                }
            }
            const float to0 = g.to[row], to1 = g.to[row + 8];
#pragma unroll
            for (int j = 0; j < XT; ++j) {
                out[j][0] *= to0;
                out[j][1] *= to0;
                out[j][2] *= to1;
                out[j][3] *= to1;
            }
            for (int kk = warp & 3; kk < 4; ++kk) {
                uint32_t a[4];
                frag_at<T * 2>(base + L::kMt, kk * 16, 2 * (warp & 3), a);
#pragma unroll
                for (int j = 0; j < XT / 2; ++j) {
                    uint32_t b[4];
                    frag_bt<PC * 2>(dyt, kk * 16, c0 + 2 * j, b);
                    mma(out[2 * j], a, b[0], b[1]);
                    mma(out[2 * j + 1], a, b[2], b[3]);
                }
            }
            const float Dh = g.D;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = row + 8 * e;
                const float d = g.d[t];
                uint16_t *dst = p.dx + (start + t) * p.dx_stride + static_cast<int64_t>(h) * p.P + sl * PC;
#pragma unroll
                for (int j = 0; j < XT; j += 2) {
                    // two lanes exchange a pair each: four columns in a row for either
                    uint32_t v[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t y =
                            *reinterpret_cast<const uint32_t *>(smem + (dyt - base) + at<PC * 2>(t, c0 + j + i) + q2 * 2);
                        v[i] = bf_pair(fmaf(Dh, bf_low(y), d * out[j + i][2 * e]),
                                       fmaf(Dh, bf_high(y), d * out[j + i][2 * e + 1]));
                    }
                    const bool odd = lane & 1;
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
                    if (t < cnt)
                        *reinterpret_cast<uint2 *>(dst + (c0 + j + odd) * 8 + (q2 & 4)) =
                            odd ? make_uint2(got, v[1]) : make_uint2(v[0], got);
                }
            }
        }
        // ---- each token's sums: NT / T threads per token add up the warps' and blocks' parts
        {
            constexpr int PER = NT / T;
            const int t = tid / PER, q = tid % PER, rb = t >> 4;
            float row = 0.f, col = 0.f, ci = 0.f, bi = 0.f;
            for (int x = q; x < 2 * rb + 2; x += PER) row += rows_s[x * T + t];
            for (int x = rb + q; x < 4; x += PER) col += cols_s[x * T + t];
#pragma unroll
            for (int x = q; x < NW; x += PER) {
                ci += int_s[x * T + t];
                bi += int_s[(NW + x) * T + t];
            }
#pragma unroll
            for (int x = 1; x < PER; x <<= 1) {
                row += __shfl_xor_sync(0xffffffffu, row, x);
                col += __shfl_xor_sync(0xffffffffu, col, x);
                ci += __shfl_xor_sync(0xffffffffu, ci, x);
                bi += __shfl_xor_sync(0xffffffffu, bi, x);
            }
            if (q == 0) {
                bi *= g.to[t];
                const float v[5] = {fmaf(-g.d[t], col, row), g.from[t] * ci, g.d[t] * bi, col + diag_s[t] + bi, diag_s[T + t]};
#pragma unroll
                for (int j = 0; j < 5; ++j) tok_s[j * T + t] = sl > 0 ? tok_s[j * T + t] + v[j] : v[j];
            }
            if (tid == 0) {
                float all = sl > 0 ? tok_s[5 * T] : 0.f;
#pragma unroll
                for (int x = 0; x < ALL; ++x) all += rs_s[x];
                tok_s[5 * T] = all;
            }
        }
    }
    if (__syncthreads_or(!ok) || s_abort) {
        // copies may still be in flight into this CTA's shared memory
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 20000000ull) {
        }
        return;
    }
    if (warp == ALL - 1) finish_head(he - 1, gates[(work / slices - 1) % 3]);
    // ---- dB and dC: this CTA's share, or the result where it has the whole group
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = m * 16 + 8 * e + gl;
            if (t >= cnt) continue;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int64_t at_n = static_cast<int64_t>(grp) * N + cw * 16 + 8 * n + q2;
                if (w.dbc) {
                    // planes: the splits' dB, then their dC
                    const int64_t plane = p.rows * p.G * N;
                    float *d = w.dbc + (split_i + (which ? 0 : w.splits)) * plane + (start + t) * p.G * N + at_n;
                    *reinterpret_cast<float2 *>(d) = make_float2(acc[m][n][2 * e], acc[m][n][2 * e + 1]);
                } else {
                    uint16_t *d = which ? p.dB + (start + t) * p.db_stride : p.dC + (start + t) * p.dc_stride;
                    *reinterpret_cast<uint32_t *>(d + at_n) = bf_pair(acc[m][n][2 * e], acc[m][n][2 * e + 1]);
                }
            }
        }
}

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
int head_splits(int64_t rows, int64_t n, int32_t H, int32_t G, int32_t N) {
    const int64_t ctas = scan_cells(rows, n, N) * G;
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
    const size_t cells = static_cast<size_t>(scan_cells(rows, n, N));
    const size_t all = cells * H * N * P * sizeof(float);
    l.splits = head_splits(rows, n, H, G, N);
    l.states = 0;
    l.grads = round256(all);
    l.dbc = l.grads + round256(all);
    l.part = l.dbc + (l.splits > 1 ? round256(2 * static_cast<size_t>(l.splits) * rows * G * N * sizeof(float)) : 0);
    l.pieces = l.part + round256(cells * 3 * H * sizeof(float));
    l.total = l.pieces + round256(scan_states_workspace_bytes(rows, n, H, P, N));
    return l;
}

cudaError_t bwd_launch(const ScanParams &p, const BwdWork &w, cudaStream_t s) {
    constexpr int bytes = BwdSmem::kBytes;
    cudaError_t err = allow_smem(scan_bwd_kernel, bytes);
    if (err != cudaSuccess) return err;
    const int64_t ctas = w.cells * p.G * w.splits;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    BwdMaps maps;
    memset(&maps, 0, sizeof(maps));
    const int64_t hp = static_cast<int64_t>(p.H) * p.P, all = w.cells * p.H * N;
    constexpr auto f32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    if (p.rows > 0 && (!tc::encode(&maps.x, p.x, hp, p.rows, p.x_stride, T) ||
                       !tc::encode(&maps.dy, p.dout, hp, p.rows, p.dout_stride, T) ||
                       !tc::encode(&maps.states, f32, 4, w.states, p.P, all, p.P, N) ||
                       !tc::encode(&maps.grads, f32, 4, w.grads, p.P, all, p.P, N)))
        return cudaErrorInvalidValue;
    scan_bwd_kernel<<<static_cast<unsigned>(ctas), 4 * N, bytes, s>>>(p, w, maps);
    return cudaGetLastError();
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
    w.cells = scan_cells(p.rows, p.seqs.n, p.N);
    cudaError_t err = launch_scan_states(p, states, grads, pieces, s);
    if (err == cudaSuccess && w.cells > 0)
        err = p.N == 128 ? launch_scan_tc_bwd(p, w, s) : bwd_launch(p, w, s);
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

cudaError_t read_and_clear_scan_bwd_error(unsigned int *value) {
    cudaError_t err = cudaMemcpyFromSymbol(value, scan::g_scan_bwd_error, sizeof(*value));
    if (err != cudaSuccess || *value == 0) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(scan::g_scan_bwd_error, &zero, sizeof(zero));
}

}  // namespace kda
