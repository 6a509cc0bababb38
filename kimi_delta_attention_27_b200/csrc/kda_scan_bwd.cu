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
// workspace: that is its bulk, and what bounds the backward's traffic. The gradient kernel then takes all
// tiles at once. One CTA of N / 8 warps has one tile of one group and walks (a share of) the group's heads,
// so C B^T is computed once, and dB and dC add up over the heads in registers, without atomics. Warp w owns
// the columns [8 w, +8) of dB and dC: S_0 and R go from memory straight into its operand fragments, the next
// head's while this one's are multiplied. Where tiles x groups leave SMs idle the heads are shared out over
// several CTAs, whose dB and dC are added by scan_bc_kernel in a fixed order. Sums over tokens go by partial sums per tile, too: runs repeat bit for bit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_scan.cuh"

namespace kda {
namespace scan {

template <int N>
struct BwdSmem {
    static constexpr int NW = N / 8;                       // warps: one per 8 columns of dB and dC
    static constexpr int kBC = T * N * 2, kX = T * PC * 2, kM = T * T * 2;
    static constexpr int kB = 0, kC = kBC;
    static constexpr int kXY = 2 * kBC;                    // two stages of x and dy
    static constexpr int kMt = kXY + 4 * kX, kKt = kMt + kM;
    static constexpr int kR = kKt + kM;                    // R in bf16, N x 64
    static constexpr int kGates = kR + N * PC * 2;
    static constexpr int kRow = kGates + 2 * static_cast<int>(sizeof(Gates));   // [8][T] row sums of M . Q d
    static constexpr int kCol = kRow + 8 * T * 4;          // [4][T] column sums of M . Q, without the diagonal
    static constexpr int kDiag = kCol + 4 * T * 4;         // [2][T] the diagonals of M . Q and of Q
    static constexpr int kInt = kDiag + 2 * T * 4;         // [2][NW][T] C . (S_0 dy) and B . (R x)
    static constexpr int kRS = kInt + 2 * NW * T * 4;      // [NW] <R, S_0>
    static constexpr int kSum = kRS + 64;                  // [11][32] the first warp's sums over a head's slices
    static constexpr int kBytes = kSum + 11 * 32 * 4;
};

// 16 x 8 blocks of the lower triangle of a 64 x 64 matrix: row block 0 has 2, 1 has 4, 2 has 6, 3 has 8
__device__ __forceinline__ void triangle_block(int j, int &rb, int &cb) {
    rb = j < 2 ? 0 : j < 6 ? 1 : j < 12 ? 2 : 3;
    cb = j - rb * (rb + 1);
}

struct BwdWork {
    const float *states, *grads;   // [cells, H, N, P]: entering states, gradients of leaving states
    float *dbc;                    // [2][splits][rows][G][N] or nullptr (one split: written to dB, dC)
    float *part;                   // [cells][3][H]: sums of d dlog a, ddt, Q_tt
    int32_t splits;
    int64_t cells;
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

template <int N>
__global__ void __launch_bounds__(4 * N, 1) scan_bwd_kernel(ScanParams p, BwdWork w) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = BwdSmem<N>;
    constexpr int NW = L::NW, NT = 32 * NW, ROWB = N * 2, BLOCKS = (20 + NW - 1) / NW, XT = 32 / NW;
    const uint32_t base = smem_addr(smem);
    Gates *gates = reinterpret_cast<Gates *>(smem + L::kGates);
    float *rows_s = reinterpret_cast<float *>(smem + L::kRow), *cols_s = reinterpret_cast<float *>(smem + L::kCol);
    float *diag_s = reinterpret_cast<float *>(smem + L::kDiag), *int_s = reinterpret_cast<float *>(smem + L::kInt);
    float *rs_s = reinterpret_cast<float *>(smem + L::kRS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gl = lane >> 2, q2 = (lane & 3) * 2;
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
    const int64_t start = u.a, sn = static_cast<int64_t>(N) * p.P;

    auto fetch = [&](int k, int stage) {
        const int64_t at_c = static_cast<int64_t>(hb + k / slices) * p.P + (k % slices) * PC;
        const uint32_t d = base + L::kXY + stage * 2 * L::kX;
        load_tile<PC * 2, NT>(d, p.x + start * p.x_stride + at_c, p.x_stride, cnt);
        load_tile<PC * 2, NT>(d + L::kX, p.dout + start * p.dout_stride + at_c, p.dout_stride, cnt);
        cp_async_commit();
    };
    load_tile<ROWB, NT>(base + L::kB, p.B + start * p.b_stride + static_cast<int64_t>(grp) * N, p.b_stride, cnt);
    load_tile<ROWB, NT>(base + L::kC, p.C + start * p.c_stride + static_cast<int64_t>(grp) * N, p.c_stride, cnt);
    fetch(0, 0);
    if (warp == 0) {
        float d0, d1;
        load_steps(p, start, cnt, hb, d0, d1);
        make_gates(gates[0], d0, d1, p.A[hb]);
    }
    cp_async_wait_all();
    __syncthreads();

    // C B^T, the blocks of the lower triangle that this warp keeps
    float cb_acc[BLOCKS][4];
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j) {
        cb_acc[j][0] = cb_acc[j][1] = cb_acc[j][2] = cb_acc[j][3] = 0.f;
        if (warp + j * NW < 20) {
            int rb, cb;
            triangle_block(warp + j * NW, rb, cb);
#pragma unroll
            for (int k = 0; k < N / 16; ++k) {
                uint32_t a[4], b[4];
                frag_a<ROWB>(base + L::kC, rb * 16, 2 * k, a);
                frag_b<ROWB>(base + L::kB, (cb >> 1) * 16, 2 * k, b);
                mma(cb_acc[j], a, cb & 1 ? b[2] : b[0], cb & 1 ? b[3] : b[1]);
            }
        }
    }
    float dc[4][4], db[4][4];   // rows 16 m, columns 8 warp
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) dc[m][j] = db[m][j] = 0.f;
    // this warp's rows of S_0 and R as B fragments ([kk]: columns 16 kk + q2, + 8), one head ahead
    float2 vs[4][2], vr[4][2];
    auto state_at = [&](const float *of, int k) {
        return of + (unit * p.H + hb + k / slices) * sn + (k % slices) * PC + static_cast<int64_t>(warp * 8 + gl) * p.P + q2;
    };
    auto load_state = [&](const float *src, float2 (&v)[4][2]) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            v[kk][0] = *reinterpret_cast<const float2 *>(src + kk * 16);
            v[kk][1] = *reinterpret_cast<const float2 *>(src + kk * 16 + 8);
        }
    };
    load_state(state_at(w.states, 0), vs);
    load_state(state_at(w.grads, 0), vr);
    float *sum_s = reinterpret_cast<float *>(smem + L::kSum);

    for (int k = 0; k < work; ++k) {
        const int h = hb + k / slices, sl = k % slices, stage = k & 1;
        const Gates &g = gates[(k / slices) & 1];
        const uint32_t xt = base + L::kXY + stage * 2 * L::kX, dyt = xt + L::kX;
        if (k > 0) {
            cp_async_wait_all();
            __syncthreads();   // x, dy, gates of this head; the other stage and all of the last head's sums are free
        }
        if (k + 1 < work) fetch(k + 1, stage ^ 1);
        // ---- Q, M, K and the sums of M . Q
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j) {
            if (warp + j * NW < 20) {
                int rb, cb;
                triangle_block(warp + j * NW, rb, cb);
                float qa[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < PC / 16; ++kk) {
                    uint32_t a[4], b[4];
                    frag_a<PC * 2>(dyt, rb * 16, 2 * kk, a);
                    frag_b<PC * 2>(xt, (cb >> 1) * 16, 2 * kk, b);
                    mma(qa, a, cb & 1 ? b[2] : b[0], cb & 1 ? b[3] : b[1]);
                }
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
        // ---- dy S_0^T and x R^T: 64 x 8 for this warp
        float rs = 0.f;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int x = 0; x < 2; ++x) rs = fmaf(vs[kk][x].x, vr[kk][x].x, fmaf(vs[kk][x].y, vr[kk][x].y, rs));
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float2(&v)[4][2] = which ? vr : vs;
            const uint32_t at_tile = which ? xt : dyt, bc = which ? L::kB : L::kC;
            float tmp[4][4];
#pragma unroll
            for (int m = 0; m < 4; ++m) tmp[m][0] = tmp[m][1] = tmp[m][2] = tmp[m][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t b[3][2];
                state_frag<3>(v[kk][0], v[kk][1], b);
                if (which) {
                    const int row = warp * 8 + gl;
                    *reinterpret_cast<uint32_t *>(smem + L::kR + at<PC * 2>(row, 2 * kk) + q2 * 2) = b[0][0];
                    *reinterpret_cast<uint32_t *>(smem + L::kR + at<PC * 2>(row, 2 * kk + 1) + q2 * 2) = b[0][1];
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t a[4];
                    frag_a<PC * 2>(at_tile, m * 16, 2 * kk, a);
#pragma unroll
                    for (int s = 2; s >= 0; --s) mma(tmp[m], a, b[s][0], b[s][1]);
                }
            }
            if (k + 1 < work) load_state(state_at(which ? w.grads : w.states, k + 1), v);
            // the dot with C's or B's own columns, and into dC or dB
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = m * 16 + 8 * e + gl;
                    const float f = which ? g.weight[t] : g.from[t];
                    const uint32_t cv = *reinterpret_cast<const uint32_t *>(smem + bc + at<ROWB>(t, warp) + q2 * 2);
                    float dot = fmaf(tmp[m][2 * e], bf_low(cv), tmp[m][2 * e + 1] * bf_high(cv));
                    float(&to)[4] = which ? db[m] : dc[m];
                    to[2 * e] = fmaf(f, tmp[m][2 * e], to[2 * e]);
                    to[2 * e + 1] = fmaf(f, tmp[m][2 * e + 1], to[2 * e + 1]);
                    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
                    dot += __shfl_xor_sync(0xffffffffu, dot, 2);
                    if ((lane & 3) == 0) int_s[(which * NW + warp) * T + t] = dot;
                }
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, x);
        if (lane == 0) rs_s[warp] = rs;
        __syncthreads();   // M, K, R and the sums are complete
        // ---- dC += K B, dB += K^T C
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint32_t bb[2], bcf[2];
            frag_bt8<ROWB>(base + L::kB, kk * 16, warp, bb);
            frag_bt8<ROWB>(base + L::kC, kk * 16, warp, bcf);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint32_t a[4];
                if (kk <= m) {
                    frag_a<T * 2>(base + L::kKt, m * 16, 2 * kk, a);
                    mma(dc[m], a, bb[0], bb[1]);
                }
                if (kk >= m) {
                    frag_at<T * 2>(base + L::kKt, kk * 16, 2 * m, a);
                    mma(db[m], a, bcf[0], bcf[1]);
                }
            }
        }
        // ---- dx: rows 16 (warp % 4), XT 8-column tiles
        {
            const int r0 = (warp & 3) * 16, c0 = (warp >> 2) * XT, row = r0 + gl;
            float acc[XT][4];
#pragma unroll
            for (int j = 0; j < XT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < N / 16; ++kk) {
                uint32_t a[4];
                frag_a<ROWB>(base + L::kB, r0, 2 * kk, a);
#pragma unroll
                for (int j = 0; j < XT / 2; ++j) {
                    uint32_t b[4];
                    frag_bt<PC * 2>(base + L::kR, kk * 16, c0 + 2 * j, b);
                    mma(acc[2 * j], a, b[0], b[1]);
                    mma(acc[2 * j + 1], a, b[2], b[3]);
                }
            }
            const float to0 = g.to[row], to1 = g.to[row + 8];
#pragma unroll
            for (int j = 0; j < XT; ++j) {
                acc[j][0] *= to0;
                acc[j][1] *= to0;
                acc[j][2] *= to1;
                acc[j][3] *= to1;
            }
            for (int kk = warp & 3; kk < 4; ++kk) {
                uint32_t a[4];
                frag_at<T * 2>(base + L::kMt, kk * 16, 2 * (warp & 3), a);
#pragma unroll
                for (int j = 0; j < XT / 2; ++j) {
                    uint32_t b[4];
                    frag_bt<PC * 2>(dyt, kk * 16, c0 + 2 * j, b);
                    mma(acc[2 * j], a, b[0], b[1]);
                    mma(acc[2 * j + 1], a, b[2], b[3]);
                }
            }
            const float Dh = p.D ? p.D[h] : 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = row + 8 * e;
                if (t < cnt) {
                    const float d = g.d[t];
                    uint16_t *dst = p.dx + (start + t) * p.dx_stride + static_cast<int64_t>(h) * p.P + sl * PC;
#pragma unroll
                    for (int j = 0; j < XT; ++j) {
                        const uint32_t y =
                            *reinterpret_cast<const uint32_t *>(smem + (dyt - base) + at<PC * 2>(t, c0 + j) + q2 * 2);
                        *reinterpret_cast<uint32_t *>(dst + (c0 + j) * 8 + q2) =
                            bf_pair(fmaf(Dh, bf_low(y), d * acc[j][2 * e]), fmaf(Dh, bf_high(y), d * acc[j][2 * e + 1]));
                    }
                }
            }
        }
        // ---- the steps' gradients, by the first warp
        if (warp == 0) {
            // per token (lane l: tokens 2l and 2l + 1): q, int, in, dd, Q_tt, and <R, S_0>, summed over slices
            float v[11];
            float rs_all = 0.f;
#pragma unroll
            for (int x = 0; x < NW; ++x) rs_all += rs_s[x];
            v[10] = rs_all;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e, rb = t >> 4;
                float row = 0.f, col = 0.f, ci = 0.f, bi = 0.f;
                for (int x = 0; x < 2 * rb + 2; ++x) row += rows_s[x * T + t];
                for (int x = rb; x < 4; ++x) col += cols_s[x * T + t];
#pragma unroll
                for (int x = 0; x < NW; ++x) {
                    ci += int_s[x * T + t];
                    bi += int_s[(NW + x) * T + t];
                }
                bi *= g.to[t];
                v[e] = fmaf(-g.d[t], col, row);
                v[2 + e] = g.from[t] * ci;
                v[4 + e] = g.d[t] * bi;
                v[6 + e] = col + diag_s[t] + bi;
                v[8 + e] = diag_s[T + t];
            }
            if (slices > 1) {
#pragma unroll
                for (int j = 0; j < 11; ++j) {
                    if (sl > 0) v[j] += sum_s[j * 32 + lane];
                    sum_s[j * 32 + lane] = v[j];
                }
            }
            if (sl == slices - 1) {
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
                const float rest = g.total * v[10];
                const float dl[2] = {suf + (before + rest), after + (v[1] + v[3]) + (before + v[4] + rest)};
                const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;
                float sa = 0.f, sb = 0.f, sd = 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * lane + e;
                    if (t < cnt) {
                        float uu;
                        step_of(p.dt[(start + t) * p.H + h], bias, 0, &uu);
                        float dd = fmaf(dl[e], A, v[6 + e]);
                        if (p.softplus) dd *= 1.f / (1.f + expf(-uu));
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
            }
        } else if (warp == 1 && sl == slices - 1 && h + 1 < he) {
            float d0, d1;
            load_steps(p, start, cnt, h + 1, d0, d1);
            make_gates(gates[(k / slices + 1) & 1], d0, d1, p.A[h + 1]);
        }
    }
    // ---- dB and dC: this CTA's share, or the result where it has the whole group
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = m * 16 + 8 * e + gl;
            if (t >= cnt) continue;
            const int64_t at_n = static_cast<int64_t>(grp) * N + warp * 8 + q2;
            if (w.dbc) {
                const int64_t plane = p.rows * p.G * N;
                float *d = w.dbc + split_i * plane + (start + t) * p.G * N + at_n;
                *reinterpret_cast<float2 *>(d) = make_float2(db[m][2 * e], db[m][2 * e + 1]);
                *reinterpret_cast<float2 *>(d + w.splits * plane) = make_float2(dc[m][2 * e], dc[m][2 * e + 1]);
            } else {
                *reinterpret_cast<uint32_t *>(p.dB + (start + t) * p.db_stride + at_n) =
                    bf_pair(db[m][2 * e], db[m][2 * e + 1]);
                *reinterpret_cast<uint32_t *>(p.dC + (start + t) * p.dc_stride + at_n) =
                    bf_pair(dc[m][2 * e], dc[m][2 * e + 1]);
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
int head_splits(int64_t rows, int64_t n, int32_t H, int32_t G) {
    const int64_t ctas = scan_cells(rows, n) * G;
    const int per_group = H / G;
    int64_t best = 0;
    int best_s = 1;
    for (int s = 1; s <= per_group && s <= 32; ++s) {
        const int per = (per_group + s - 1) / s;
        if ((per_group + per - 1) / per != s) continue;   // a CTA without a head
        const int64_t cost = (ctas * s + 147) / 148 * per;
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

template <int N>
cudaError_t bwd_launch(const ScanParams &p, const BwdWork &w, cudaStream_t s) {
    constexpr int bytes = BwdSmem<N>::kBytes;
    cudaError_t err = allow_smem(scan_bwd_kernel<N>, bytes);
    if (err != cudaSuccess) return err;
    const int64_t ctas = w.cells * p.G * w.splits;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    scan_bwd_kernel<N><<<static_cast<unsigned>(ctas), 4 * N, bytes, s>>>(p, w);
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
    w.cells = scan_cells(p.rows, p.seqs.n);
    cudaError_t err = launch_scan_states(p, states, grads, pieces, s);
    if (err == cudaSuccess && w.cells > 0)
        err = by_state(p.N, [&](auto n) { return bwd_launch<decltype(n)::value>(p, w, s); });
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
