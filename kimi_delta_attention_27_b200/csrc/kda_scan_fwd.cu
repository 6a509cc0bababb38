// kda_scan_fwd.cu -- selective state space scan over prompts, sm_100a.
//
// Per sequence and head, with d_t the step, a_t = exp(d_t A) and a state S of N x P:
//
//   S_t = a_t S_{t-1} + d_t B_t x_t^T,      y_t = S_t^T C_t + D x_t.
//
// Over a tile of 64 tokens that enters with the state S_0 this is, with Gamma_t = sum of the tile's log a
// through t and L_ts = exp(Gamma_t - Gamma_s) for s <= t (else 0):
//
//   y = (L . (C B^T)) Diag(d) x + Diag(e^Gamma) C S_0 + D x,
//   S_end = e^(Gamma_end) S_0 + B^T Diag(d e^(Gamma_end - Gamma)) x,
//
// four small matrix products on the tensor cores. The operands that are inputs (x, B, C) are exact in bf16.
// The others are rounded where y, itself bf16, takes them in: L . (C B^T) d and the copy of S_0 that
// multiplies C, one rounding each. The state itself is carried in fp32, and B^T's weighted rows go in as
// two or three bf16 parts that add up to 16 or 24 bits: three where a final state is returned in fp32.
//
// One CTA of 4 warps runs the tiles of a piece of one sequence in order, for one head and 64 of its P
// columns (columns do not mix). Warp w has 16 rows of y and N / 4 rows of the state, whose accumulators stay
// in its registers from tile to tile; L . (C B^T) never leaves registers either: the accumulator layout of
// C B^T is the operand layout of the product with x. The next tile's x, B, C arrive by cp.async meanwhile.
// It is this kernel for a state size of 64, and for short sequences at 128; others take kda_scan_tc.cu. Bound by the
// latency of a tile's chain: one sequence of 200 tokens x 32 heads, four tiles, 19 us.
//
// Few long sequences make few CTAs. Then sequences are cut into pieces of whole tiles: a first launch
// (kda_scan_tc_state.cu) finds each piece's own contribution to the state it leaves (from zero), scan_join_kernel adds those up
// along each sequence, and the main launch runs all pieces at once from the states they enter with. Pieces
// lie on a global grid of `seg` tokens, so sequence i's piece in cell c has number i + c, no matter how
// the lengths fall, and a CTA finds its sequence by one search.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_scan.cuh"

namespace kda {
namespace scan {

__device__ unsigned int g_scan_error = 0;

constexpr int NT = 128;

// acc (rows [n0, + 16 MT) of the state, 64 columns) += rows^T Diag(weight) x, the weighted rows in S parts
template <int ROWB, int MT, int S>
__device__ __forceinline__ void add_outer(float (&acc)[MT][8][4], uint32_t rows_tile, uint32_t x_tile, const float *weight,
                                          int n0) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int kk = 0; kk < T / 16; ++kk) {
        uint32_t a[MT][S][4];
        const float2 w0 = *reinterpret_cast<const float2 *>(weight + kk * 16 + (lane & 3) * 2);
        const float2 w1 = *reinterpret_cast<const float2 *>(weight + kk * 16 + 8 + (lane & 3) * 2);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            uint32_t f[4];
            frag_at<ROWB>(rows_tile, kk * 16, (n0 >> 3) + 2 * m, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 w = j < 2 ? w0 : w1;
                uint32_t part[S];
                split<S>(bf_low(f[j]) * w.x, bf_high(f[j]) * w.y, part);
#pragma unroll
                for (int s = 0; s < S; ++s) a[m][s][j] = part[s];
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t b[4];
            frag_bt<PC * 2>(x_tile, kk * 16, 2 * c, b);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int s = S - 1; s >= 0; --s) {
                    mma(acc[m][2 * c], a[m][s], b[0], b[1]);
                    mma(acc[m][2 * c + 1], a[m][s], b[2], b[3]);
                }
        }
    }
}

// acc = total acc + rows^T Diag(weight) x, the tile's share added up by itself: the tensor cores cut a sum off at its last
// bit, twelve times a tile (final states of 200 tokens to 64 bits: 1e-6 without, 1e-7 with)
template <int ROWB, int MT, int S>
__device__ __forceinline__ void add_tile(float (&acc)[MT][8][4], float total, uint32_t rows_tile, uint32_t x_tile,
                                         const float *weight, int n0) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        float share[1][8][4];
#pragma unroll
        for (int c = 0; c < 8; ++c) share[0][c][0] = share[0][c][1] = share[0][c][2] = share[0][c][3] = 0.f;
        add_outer<ROWB, 1, S>(share, rows_tile, x_tile, weight, n0 + 16 * m);
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][c][e] = fmaf(acc[m][c][e], total, share[0][c][e]);
    }
}

template <int MT>
__device__ __forceinline__ void scale_state(float (&acc)[MT][8][4], float f) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][c][j] *= f;
}

// a warp's rows of a state [N, P] in memory (fp32 or bf16; null: zeros) to and from its accumulators;
// `p` at the slice's first column
template <int MT>
__device__ __forceinline__ void read_state(float (&acc)[MT][8][4], const void *state, int64_t off, bool fp32, int P, int n0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float2 v = make_float2(0.f, 0.f);
                const int64_t e = off + static_cast<int64_t>(n0 + 16 * m + 8 * j + g) * P + 8 * c + t;
                if (state) {
                    if (fp32) {
                        v = *reinterpret_cast<const float2 *>(static_cast<const float *>(state) + e);
                    } else {
                        const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(state) + e);
                        v = make_float2(bf_low(w), bf_high(w));
                    }
                }
                acc[m][c][2 * j] = v.x;
                acc[m][c][2 * j + 1] = v.y;
            }
}
template <int MT>
__device__ __forceinline__ void write_state(const float (&acc)[MT][8][4], void *state, int64_t off, bool fp32, int P,
                                            int n0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t e = off + static_cast<int64_t>(n0 + 16 * m + 8 * j + g) * P + 8 * c + t;
                if (fp32)
                    *reinterpret_cast<float2 *>(static_cast<float *>(state) + e) =
                        make_float2(acc[m][c][2 * j], acc[m][c][2 * j + 1]);
                else
                    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(state) + e) =
                        bf_pair(acc[m][c][2 * j], acc[m][c][2 * j + 1]);
            }
}

template <int N>
struct FwdSmem {
    static constexpr int kBC = T * N * 2, kX = T * PC * 2;
    static constexpr int kStage = 2 * kBC + kX;
    static constexpr int kState = 2 * kStage;                 // N x 64 bf16: the state as an operand
    static constexpr int kY = kState + N * PC * 2;
    static constexpr int kGates = kY + kX;
    static constexpr int kBytes = kGates + 2 * static_cast<int>(sizeof(Gates));
};

template <int N, int S>
__global__ void __launch_bounds__(NT, 2) scan_fwd_kernel(ScanParams p, int64_t seg, const float *entering) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = FwdSmem<N>;
    constexpr int MT = N / 64, ROWB = N * 2, KN = N / 16;
    Gates *gates = reinterpret_cast<Gates *>(smem + L::kGates);
    const uint32_t base = smem_addr(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slices = p.P / PC, hs = static_cast<int>(blockIdx.x % (p.H * slices));
    const int h = hs / slices, col = (hs % slices) * PC;
    const int64_t unit = blockIdx.x / (p.H * slices);
    if (blockIdx.x == 0) check_offsets(p.seqs, &g_scan_error);
    const Piece u = find_piece(p.seqs, unit, seg);
    if (u.none) return;
    // 16-row blocks of y have 1 to 4 blocks of C B^T to do: which warp (and so which scheduler) has the
    // longest differs from CTA to CTA. The one with the shortest makes the next tile's gates.
    const int rb = (warp + blockIdx.x) & 3;
    const int n0 = warp * (N / 4);
    const uint16_t *xs = p.x + static_cast<int64_t>(h) * p.P + col;
    const uint16_t *Bs = p.B + static_cast<int64_t>(h / (p.H / p.G)) * N;
    const uint16_t *Cs = p.C + static_cast<int64_t>(h / (p.H / p.G)) * N;
    const float A = p.A[h], Dh = p.D ? p.D[h] : 0.f;
    const int64_t sn = static_cast<int64_t>(N) * p.P;

    float acc[MT][8][4];
    if (entering)
        read_state<MT>(acc, entering, (unit * p.H + h) * sn + col, true, p.P, n0);
    else
        read_state<MT>(acc, p.h0, (static_cast<int64_t>(u.i) * p.H + h) * sn + col, p.h0_fp32, p.P, n0);

    const int64_t c_first = u.a / T, c_end = u.b > u.a ? (u.b + T - 1) / T : c_first;
    auto fetch = [&](int64_t c, int stage) {
        const int64_t s = tile_start(u, c);
        const int cnt = tile_count(u, c);
        const uint32_t d = base + stage * L::kStage;
        load_tile<ROWB, NT>(d, Cs + s * p.c_stride, p.c_stride, cnt);
        load_tile<ROWB, NT>(d + L::kBC, Bs + s * p.b_stride, p.b_stride, cnt);
        load_tile<PC * 2, NT>(d + 2 * L::kBC, xs + s * p.x_stride, p.x_stride, cnt);
        cp_async_commit();
    };
    // the state as a bf16 operand, rows of this warp
    auto publish = [&]() {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = n0 + 16 * m + 8 * j + g;
                    *reinterpret_cast<uint32_t *>(smem + L::kState + at<PC * 2>(r, c) + 4 * t) =
                        bf_pair(acc[m][c][2 * j], acc[m][c][2 * j + 1]);
                }
    };
    float d0 = 0.f, d1 = 0.f;   // the steps of the tile whose gates are made next (warp rb == 0)
    if (c_first < c_end) {
        fetch(c_first, 0);
        publish();
        if (rb == 0) {
            load_steps(p, tile_start(u, c_first), tile_count(u, c_first), h, d0, d1);
            make_gates(gates[c_first & 1], d0, d1, tile_count(u, c_first), A);
            if (c_first + 1 < c_end) load_steps(p, tile_start(u, c_first + 1), tile_count(u, c_first + 1), h, d0, d1);
        }
    }
    int stage = 0;
    for (int64_t c = c_first; c < c_end; ++c, stage ^= 1) {
        cp_async_wait_all();
        __syncthreads();   // the tile, its gates and the state's copy are there; the other stage is free
        if (c + 1 < c_end) fetch(c + 1, stage ^ 1);
        if (rb == 0 && c + 1 < c_end) {
            make_gates(gates[(c + 1) & 1], d0, d1, tile_count(u, c + 1), A);
            if (c + 2 < c_end) load_steps(p, tile_start(u, c + 2), tile_count(u, c + 2), h, d0, d1);
        }
        const Gates &g = gates[c & 1];
        const uint32_t ct = base + stage * L::kStage, bt = ct + L::kBC, xt = bt + L::kBC, st = base + L::kState;
        const int cnt = tile_count(u, c), r0 = rb * 16, row = r0 + (lane >> 2), q = (lane & 3) * 2;
        const int64_t start = tile_start(u, c);
        if (r0 < cnt) {
            float y[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j][0] = y[j][1] = y[j][2] = y[j][3] = 0.f;
            uint32_t ca[KN][4];
#pragma unroll
            for (int k = 0; k < KN; ++k) {
                frag_a<ROWB>(ct, r0, 2 * k, ca[k]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t b[4];
                    frag_bt<PC * 2>(st, k * 16, 2 * j, b);
                    mma(y[2 * j], ca[k], b[0], b[1]);
                    mma(y[2 * j + 1], ca[k], b[2], b[3]);
                }
            }
            const float f0 = g.from[row], f1 = g.from[row + 8];
            const float h0 = g.hi[row], h1 = g.hi[row + 8], l0 = g.lo[row], l1 = g.lo[row + 8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j][0] *= f0;
                y[j][1] *= f0;
                y[j][2] *= f1;
                y[j][3] *= f1;
            }
            for (int sb = 0; sb <= rb; ++sb) {
                float m[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int k = 0; k < KN; ++k) {
                    uint32_t b[4];
                    frag_b<ROWB>(bt, sb * 16, 2 * k, b);
                    mma(m[0], ca[k], b[0], b[1]);
                    mma(m[1], ca[k], b[2], b[3]);
                }
                uint32_t a[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int s = sb * 16 + 8 * j + q;
                    const float2 hs2 = *reinterpret_cast<const float2 *>(&g.hi[s]);
                    const float2 ls2 = *reinterpret_cast<const float2 *>(&g.lo[s]);
                    const float2 ds2 = *reinterpret_cast<const float2 *>(&g.d[s]);
                    const float m0 = m[j][0] * ds2.x * ex2((h0 - hs2.x) + (l0 - ls2.x));
                    const float m1 = m[j][1] * ds2.y * ex2((h0 - hs2.y) + (l0 - ls2.y));
                    const float m2 = m[j][2] * ds2.x * ex2((h1 - hs2.x) + (l1 - ls2.x));
                    const float m3 = m[j][3] * ds2.y * ex2((h1 - hs2.y) + (l1 - ls2.y));
                    a[2 * j] = bf_pair(s <= row ? m0 : 0.f, s + 1 <= row ? m1 : 0.f);
                    a[2 * j + 1] = bf_pair(s <= row + 8 ? m2 : 0.f, s + 1 <= row + 8 ? m3 : 0.f);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t b[4];
                    frag_bt<PC * 2>(xt, sb * 16, 2 * j, b);
                    mma(y[2 * j], a, b[0], b[1]);
                    mma(y[2 * j + 1], a, b[2], b[3]);
                }
            }
            // D x, then the warp's 16 rows by way of shared memory, for 16-byte stores
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t x0 = *reinterpret_cast<const uint32_t *>(smem + (xt - base) + at<PC * 2>(row, j) + 2 * q);
                const uint32_t x1 =
                    *reinterpret_cast<const uint32_t *>(smem + (xt - base) + at<PC * 2>(row + 8, j) + 2 * q);
                *reinterpret_cast<uint32_t *>(smem + L::kY + at<PC * 2>(row, j) + 2 * q) =
                    bf_pair(fmaf(Dh, bf_low(x0), y[j][0]), fmaf(Dh, bf_high(x0), y[j][1]));
                *reinterpret_cast<uint32_t *>(smem + L::kY + at<PC * 2>(row + 8, j) + 2 * q) =
                    bf_pair(fmaf(Dh, bf_low(x1), y[j][2]), fmaf(Dh, bf_high(x1), y[j][3]));
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = r0 + j * 4 + (lane >> 3), ch = lane & 7;
                if (r < cnt)
                    *reinterpret_cast<uint4 *>(p.out + (start + r) * p.out_stride + static_cast<int64_t>(h) * p.P + col +
                                               ch * 8) =
                        *reinterpret_cast<const uint4 *>(smem + L::kY + at<PC * 2>(r, ch));
            }
        }
        if (c + 1 < c_end || (u.last && p.hT)) {
            if constexpr (S == 3) {
                add_tile<ROWB, MT, S>(acc, g.total, bt, xt, g.weight, n0);
            } else {
                scale_state<MT>(acc, g.total);
                add_outer<ROWB, MT, S>(acc, bt, xt, g.weight, n0);
            }
            __syncthreads();   // every warp has read the state's copy
            if (c + 1 < c_end) publish();
        }
    }
    if (u.last && p.hT)
        write_state<MT>(acc, p.hT, (static_cast<int64_t>(u.i) * p.H + h) * sn + col, p.hT_fp32, p.P, n0);
}

// Along every sequence: pieces' own contributions become the states they enter with, in place:
// S = init;  for each piece: (its contribution, S) <- (S, decay S + contribution).
// grid (sequences * H, elements / 1024): a thread has four elements of the state.
template <bool kReverse>
__global__ void __launch_bounds__(256) scan_join_kernel(ScanParams p, int64_t seg, float *ws, const float *decay) {
    const int64_t ih = blockIdx.x;
    const int32_t i = static_cast<int32_t>(ih / p.H), h = static_cast<int32_t>(ih % p.H);
    const int64_t sn = static_cast<int64_t>(p.N) * p.P, e = (static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x) * 4;
    if (e >= sn) return;
    const int64_t c0 = cell_of(p.seqs.begin(i), seg), c1 = cell_of(p.seqs.end(i), seg);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const void *init = kReverse ? static_cast<const void *>(p.dhT) : p.h0;
    if (init) {
        if (kReverse || p.h0_fp32) {
            s = *reinterpret_cast<const float4 *>(static_cast<const float *>(init) + ih * sn + e);
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(init) + ih * sn + e);
            s = make_float4(bf_low(w.x), bf_high(w.x), bf_low(w.y), bf_high(w.y));
        }
    }
    const int64_t count = c1 - c0 + 1;
    constexpr int U = 4;
    for (int64_t k0 = 0; k0 < count; k0 += U) {
        // the contributions do not depend on one another: four loads at once, then the chain
        float4 v[U];
        float f[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            f[j] = 0.f;
            if (k0 + j + 1 < count) {   // what the last piece adds is not needed
                const int64_t unit = i + (kReverse ? c1 - k0 - j : c0 + k0 + j);
                v[j] = *reinterpret_cast<const float4 *>(ws + (unit * p.H + h) * sn + e);
                f[j] = decay[unit * p.H + h];
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k0 + j < count) {
                const int64_t unit = i + (kReverse ? c1 - k0 - j : c0 + k0 + j);
                *reinterpret_cast<float4 *>(ws + (unit * p.H + h) * sn + e) = s;
                s = make_float4(fmaf(f[j], s.x, v[j].x), fmaf(f[j], s.y, v[j].y), fmaf(f[j], s.z, v[j].z),
                                fmaf(f[j], s.w, v[j].w));
            }
        }
    }
}

// Tokens per piece, a multiple of `tile`; 0: whole sequences. `ctas`: CTAs of one piece, `slots` as many as run at
// once. Whole sequences take as long as the longest; a cut costs a second reading of x and B, one state per piece and
// two more launches, 1.5 times the work where the pieces are long and over twice that where they are not. So sequences
// are cut where equal ones fill less than half of the slots, and packed ones, of which the longest is taken to be twice
// the mean, fewer than all. (4096 tokens x 64 heads x 64: 2 sequences, 64 CTAs, 176 us whole, 181 cut; 3 sequences 181
// and 231. One of 65536 tokens x 32 heads x 128, 32 CTAs: 2.62 ms whole, 0.86 cut. 2 packed ones, 13493
// tokens x 64 heads x 64, 64 CTAs: 286 and 244.) And only where the longest makes two pieces and has `least` tokens:
// below that the launches cost more than the pieces save. (32 heads x 64, state size 128, us whole and cut: 2 rows of 200
// tokens 25 and 41, of 400 33 and 45, of 600 43 and 46, of 800 49 and 43; state size 64: 21 and 31, 31 and 33, 41 and 37,
// 51 and 37.)
int64_t piece_tokens(int64_t rows, int64_t n, bool packed, int64_t ctas, int slots, int tile, int64_t least) {
    if (n == 0 || (packed ? 1 : 2) * n * ctas >= slots) return 0;
    const int64_t want = 2 * slots, longest = packed && n > 1 ? 2 * rows / n : rows / n;
    int64_t seg = (rows * ctas + want - 1) / want;
    seg = (seg + tile - 1) / tile * tile;
    if (seg < 256) seg = 256;
    return longest < 2 * seg || longest < least ? 0 : seg;
}
// State size 128: the tcgen05 kernel takes sequences of more than 160 tokens on average, or, where the CTAs of the
// warp-level one fit the SMs at once, of more than 256: a first tile takes it some 3 us longer. (16 sequences x 64 heads:
// of 140 tokens 63 us against 61, of 180 68 and 71, of 256 60 and 85, of 512 100 and 166; one of 200 x 32: 22 and 19.)
bool takes_tc(int64_t rows, int64_t n, int64_t columns, int32_t N) {
    return N == 128 && rows > (n * columns > 2 * 148 ? 160 : 256) * n;
}
int64_t fwd_piece_tokens(int64_t rows, int64_t n, bool packed, int32_t H, int32_t P, int32_t N) {
    const int64_t columns = static_cast<int64_t>(H) * (P / PC);
    return takes_tc(rows, n, columns, N) ? piece_tokens(rows, n, packed, (columns + 1) / 2, 148, kScanTcTile, 512)
                                         : piece_tokens(rows, n, packed, columns, 2 * 148, T, 512);
}
// The backward's runs of the state, both directions at once; their tiles take so little that packed sequences, too, are
// cut only below half of the slots (the gradients of 2 packed ones, 13493 tokens x 64 heads, with tiles of 64 tokens: 656
// us whole, 827 cut), and from 1024 tokens on (8 heads x 64, state size 128, the gradients whole and cut: 2 rows of 200
// tokens 51 and 64 us, of 600 61 and 66, of 1200 80 and 72).
int64_t state_piece_tokens(int64_t rows, int64_t n, bool packed, int32_t H, int32_t P) {
    const int64_t columns = static_cast<int64_t>(H) * (P / PC), ctas = (columns + 1) / 2 * 2;
    return 2 * n * ctas >= 148 ? 0 : piece_tokens(rows, n, packed, ctas, 148, kScanTcTile, 1024);
}

int64_t piece_count(int64_t rows, int64_t n, int64_t seg) { return seg ? rows / seg + n : n; }

size_t piece_bytes(int64_t rows, int64_t n, int64_t seg, int32_t H, int32_t P, int32_t N) {
    if (!seg) return 0;
    return static_cast<size_t>(piece_count(rows, n, seg)) * H * (static_cast<size_t>(N) * P + 4) * sizeof(float);
}

template <bool kReverse>
cudaError_t join_launch(const ScanParams &p, int64_t seg, float *ws, const float *decay, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(p.seqs.n) * p.H),
                    static_cast<unsigned>((static_cast<int64_t>(p.N) * p.P + 1023) / 1024));
    scan_join_kernel<kReverse><<<grid, 256, 0, s>>>(p, seg, ws, decay);
    return cudaGetLastError();
}

}  // namespace scan

// the larger need, that of packed sequences: where equal ones are cut, those are too
size_t scan_fwd_workspace_bytes(int64_t rows, int64_t n, int32_t H, int32_t P, int32_t N) {
    return scan::piece_bytes(rows, n, scan::fwd_piece_tokens(rows, n, true, H, P, N), H, P, N);
}

size_t scan_states_workspace_bytes(int64_t rows, int64_t n, int32_t H, int32_t P, int32_t N) {
    // both directions' pieces; the larger need again
    return 2 * scan::piece_bytes(rows, n, scan::state_piece_tokens(rows, n, true, H, P), H, P, N);
}

template <int N>
cudaError_t scan_fwd_launch(const ScanParams &p, int64_t seg, int64_t units, const float *entering, cudaStream_t s) {
    using namespace scan;
    auto *k = p.hT && p.hT_fp32 ? scan_fwd_kernel<N, 3> : scan_fwd_kernel<N, 2>;
    const cudaError_t err = allow_smem(k, FwdSmem<N>::kBytes);
    if (err != cudaSuccess) return err;
    k<<<static_cast<unsigned>(units * p.H * (p.P / PC)), NT, FwdSmem<N>::kBytes, s>>>(p, seg, entering);
    return cudaGetLastError();
}

cudaError_t launch_scan_fwd(const ScanParams &p, cudaStream_t s) {
    using namespace scan;
    const int64_t cut = fwd_piece_tokens(p.rows, p.seqs.n, p.seqs.cu != nullptr, p.H, p.P, p.N);
    const int64_t seg = cut ? cut : kWhole, units = piece_count(p.rows, p.seqs.n, cut);
    if (units * p.H * (p.P / PC) > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (cut) {
        float *decay = p.ws + units * p.H * p.N * p.P;
        cudaError_t err = launch_scan_tc_state(p, p.hT && p.hT_fp32 ? 3 : 2, 1, seg, units, {nullptr, p.ws, decay, nullptr}, {}, s);
        if (err == cudaSuccess) err = join_launch<false>(p, seg, p.ws, decay, s);
        if (err != cudaSuccess) return err;
    }
    const float *entering = cut ? p.ws : nullptr;
    if (takes_tc(p.rows, p.seqs.n, static_cast<int64_t>(p.H) * (p.P / PC), p.N)) return launch_scan_tc(p, seg, units, entering, s);
    return by_state(p.N, [&](auto n) { return scan_fwd_launch<decltype(n)::value>(p, seg, units, entering, s); });
}

cudaError_t launch_scan_states(const ScanParams &p, float *states, float *grads, float *ws, cudaStream_t s) {
    using namespace scan;
    const int64_t cut = state_piece_tokens(p.rows, p.seqs.n, p.seqs.cu != nullptr, p.H, p.P), seg = cut ? cut : kWhole;
    const int64_t units = piece_count(p.rows, p.seqs.n, cut);
    if (units == 0) return cudaSuccess;
    if (units * p.H * (p.P / PC) > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int64_t all = units * p.H * p.N * p.P;
    float *wf = ws, *df = wf + all, *wr = df + 4 * units * p.H, *dr = wr + all;
    auto run = [&](bool local) {
        const ScanStateRun f = local ? ScanStateRun{nullptr, wf, df, nullptr} : ScanStateRun{cut ? wf : nullptr, nullptr, nullptr, states};
        const ScanStateRun r = local ? ScanStateRun{nullptr, wr, dr, nullptr} : ScanStateRun{cut ? wr : nullptr, nullptr, nullptr, grads};
        return launch_scan_tc_state(p, 3, 2, seg, units, f, r, s);
    };
    cudaError_t err = cudaSuccess;
    if (cut) {
        err = run(true);
        if (err == cudaSuccess) err = join_launch<false>(p, seg, wf, df, s);
        if (err == cudaSuccess) err = join_launch<true>(p, seg, wr, dr, s);
    }
    return err == cudaSuccess ? run(false) : err;
}

cudaError_t read_and_clear_scan_error(unsigned int *value) {
    cudaError_t err = cudaMemcpyFromSymbol(value, scan::g_scan_error, sizeof(*value));
    if (err != cudaSuccess || *value == 0) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(scan::g_scan_error, &zero, sizeof(zero));
}

}  // namespace kda
