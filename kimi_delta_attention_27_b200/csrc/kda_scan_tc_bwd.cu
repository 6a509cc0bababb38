// kda_scan_tc_bwd.cu -- gradients of the selective state space scan on tcgen05, state sizes 64 and 128, sm_100a.
//
// The formulas are those of kda_scan_bwd.cu, with tiles of 128 tokens and the products between tokens transposed, so
// that a thread has one row s of them and the sums over t that make dB and dx need no transposed operand:
//
//   Gt = B C^T, Qt = x dy^T                           128 x 128 (s, t); Gt once for all heads of a group
//   Mt = L^T . Gt,  Kt = L^T . Qt Diag(d_s)           in bf16, zero for t < s
//   Y  = C S_0,  Z = B R                              128 x 64, S_0 and R in three bf16 parts
//   dC += K B + (e^Gamma dy) S_0^T                    128 x 128, over the heads, S_0 and R in two parts
//   dB += Kt C + (d e^(Gamma_end - Gamma) x) R^T
//   dx = Diag(d) (Mt dy) + Diag(d e^(Gamma_end - Gamma)) Z + D dy
//
// and the steps' gradients from the elementwise Mt . Qt, the dots dy_t . Y_t and x_s . Z_s, and <R, S_0>.
// Mt is the first operand of its product from TMEM; Kt lies in shared memory once and is read as K and as its transpose.
// dB and dC stay in TMEM over all of a CTA's heads.
//
// At a state size of 128 the products take some 4900 cycles per tile and head (operands from shared memory, 128 bytes a
// cycle), the elements' own traffic with shared memory and TMEM 4700 more, the states' 64 KB some 2800 at HBM's rate, the elements'
// instructions 5200 of each scheduler. Sixteen warps do the elements: they turn S_0 into parts, then, while its products
// run, form Mt and Kt, then turn R into parts in the same place. One warp issues the products and loads; one makes the
// gates of the next head and finishes the sums of the last. What is left is the chain of those phases: 2 x 4096 tokens x
// 64 heads x 64 take 264 us, 13500 cycles per tile and head, tensor cores 34 % and the L1 pipes 49 % busy. (Warp-level
// products with tiles of 64 tokens: 536 us. R taken in between the two halves of Mt and Kt, so that its products run
// under the second: 280 us. States loaded to registers rather than by TMA: 422 us.) At 64: 5 packed sequences, 3802
// tokens x 32 heads x 128, 2 groups: 129 us.
//
// Every wait is bounded; one that runs out raises kErrTimeout and winds the CTA down.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_scan_tc.cuh"

namespace kda {
namespace scan {
namespace tc {

__device__ unsigned int g_scan_tc_bwd_error = 0;
#ifdef KDA_TEST_HOOKS
// Test-only build (never the product library): the gates of this head of every CTA are not signalled, so that the bounded
// waits for them run out.
__device__ int g_scan_tc_bwd_stall = -1;
#endif

constexpr int TT = kScanTcTile;
constexpr int kIssuer = 16, NT = 32 * 18;   // warp 17: gates and sums

struct HeadGates {
    float hi[TT], lo[TT];   // log2 of the decay from the tile's start through token t, in two floats
    float d[TT];            // the steps
    float from[TT];         // e^Gamma
    float to[TT];           // e^(Gamma_end - Gamma)
    float weight[TT];       // d to
    float slope[TT];        // of the step in dt
    float col[TT];          // decay from the start of the token's quarter through it
    float open_hi[4], open_lo[4];   // Gamma at the quarters' starts
    float total, A, D;
    uint32_t steep;         // bit c: the decays within quarter c span more than 2^60, down or up
};

// sums over parts of the tile, for the helper: [which][token]
struct Partials {
    float row[4][TT];       // sums over the 32 tokens of a quarter of Mt . Qt d
    float col[4][TT];       // and of Mt . Qt, without the diagonal
    float leave[4][TT];     // dy . Y over 16 columns
    float enter[4][TT];     // x . Z
    float near[TT];         // of Mt . Qt d over the token's own quarter
    float diag[TT], q[TT];  // the diagonals of Mt . Qt and of Qt
    float rs[16];           // <R, S_0>
};

// NS: state size
template <int NS>
struct BwdSmem {
    static constexpr uint32_t kTile = NS / 64 * kBlock;                    // B or C: blocks of 64 columns
    static constexpr uint32_t kPart = NS * 128;                            // a part of a state: rows of 64 columns
    static constexpr uint32_t kC = 0, kB = kTile;
    static constexpr uint32_t kXY = 2 * kTile;               // [stage] x and dy; before them, the last head's R
    static constexpr uint32_t kParts = kXY + 4 * kBlock;     // three parts of S_0, then of R
    static constexpr uint32_t kK = kParts + 3 * kPart;       // S_0, then Kt: two blocks of columns
    static constexpr uint32_t kGates = kK + 2 * kBlock;                    // [2]
    static constexpr uint32_t kSums = kGates + 2 * sizeof(HeadGates);
    static constexpr uint32_t kBars = kSums + sizeof(Partials);
    static constexpr uint32_t kBytes = kBars + 8 * 22;
    static_assert(kBytes + 64 <= 227 * 1024, "shared memory of one CTA");
};

// TMEM columns. Mt takes the first half of Qt's place once that has been read, Mt dy the second; Z takes Y's.
constexpr uint32_t kColDc = 0, kColDb = 128, kColQ = 256, kColM = 256, kColX = 320, kColY = 384, kColDy = 448, kColSx = 480;

constexpr uint32_t kIdQ = idesc_f16(128, 128, 1, 0, 0);    // both K-major
constexpr uint32_t kIdY = idesc_f16(128, 64, 1, 0, 1);     // K-major, MN-major

struct BwdMaps {
    CUtensorMap x, dy, b, c, states, grads;
};

// barriers; those from kByAll on are arrived at by each of the sixteen warps
enum : int {
    kBcFull = 0,
    kXFull = 1,       // [stage] x and dy
    kSFull = 3,       // S_0
    kRFull = 4,       // R
    kQ = 5,           // Qt (first: Gt) is there
    kSDone = 6,       // the products with S_0 are done
    kZ = 7,           // Z and Mt dy are there
    kEnd = 8,         // all products of the head are done
    kGatesFull = 9,   // [2]
    kSumsFree = 11,   // the helper has read a head's sums
    kByAll = 12,
    kQReady = 12,     // the place of Qt is free, x and dy end in zeros
    kSParts = 13,     // S_0's parts and the scaled rows are written, the last head's x and dy used
    kRParts = 14,     // R's parts are written
    kMk = 15,         // Mt and Kt are written
    kSums = 16,       // a head's sums are written
    kQRead = 17,      // [quarter] its four warps have read Qt
    kBarCount = 21
};

// The gates of a head, by one warp: lane l has tokens 4 l .. 4 l + 3 (u: their steps before softplus).
__device__ __forceinline__ void make_head_gates(HeadGates &g, const float (&dt)[4], int cnt, float A, float bias, float D,
                                                int softplus) {
    const int lane = threadIdx.x & 31;
    const Two a2 = log2_rate(A);
    float d[4], slope[4];
    Two c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float u;
        d[j] = step_of(dt[j], bias, softplus, &u);
        if (4 * lane + j >= cnt) d[j] = 0.f;
        slope[j] = softplus ? 1.f / (1.f + expf(-u)) : 1.f;
        c[j] = 4 * lane + j < cnt ? log_decay(d[j], a2) : Two{0.f, 0.f};
        if (j) c[j] = c[j - 1] + c[j];
    }
    const Two s = scan_lanes(c[3]), total = shfl(s, 31);
    Two before = {__shfl_up_sync(0xffffffffu, s.hi, 1), __shfl_up_sync(0xffffffffu, s.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const Two opens = shfl(before, lane & 24), closes = shfl(s, lane | 7);   // the quarter's start and end
    float hi[4], lo[4], from[4], to[4], col[4];
    const float whole = minus(opens, closes);
    float span = fabsf(whole);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const Two v = before + c[j];
        hi[j] = v.hi;
        lo[j] = v.lo;
        from[j] = ex2(v);
        to[j] = ex2(minus(total, v));
        const float from_start = minus(v, opens);
        span = fmaxf(span, fabsf(from_start));
        col[j] = ex2(from_start);
    }
    // by eight lanes of a quarter each; a NaN counts, for it must reach no token that does not depend on it
    const unsigned steep = __ballot_sync(0xffffffffu, span > 60.f || isnan(whole));
    auto put = [&](float *dst, float a, float b, float e, float f) {
        reinterpret_cast<float4 *>(dst)[lane] = make_float4(a, b, e, f);
    };
    put(g.hi, hi[0], hi[1], hi[2], hi[3]);
    put(g.lo, lo[0], lo[1], lo[2], lo[3]);
    put(g.d, d[0], d[1], d[2], d[3]);
    put(g.from, from[0], from[1], from[2], from[3]);
    put(g.to, to[0], to[1], to[2], to[3]);
    put(g.weight, d[0] * to[0], d[1] * to[1], d[2] * to[2], d[3] * to[3]);
    put(g.slope, slope[0], slope[1], slope[2], slope[3]);
    put(g.col, col[0], col[1], col[2], col[3]);
    if ((lane & 7) == 0) {
        g.open_hi[lane >> 3] = opens.hi;
        g.open_lo[lane >> 3] = opens.lo;
    }
    if (lane == 0) {
        g.total = ex2(total);
        g.A = A;
        g.D = D;
        g.steep = steep_blocks(steep);
    }
}

// The sums over a warp's lanes of 16 values: lane l returns that of v[l % 16].
__device__ __forceinline__ float sum_lanes16(float (&v)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float send = up ? v[i] : v[i + m], keep = up ? v[i + m] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

template <int NS>
__global__ void __launch_bounds__(NT, 1) scan_tc_bwd_kernel(ScanParams p, BwdWork w, const __grid_constant__ BwdMaps maps) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = BwdSmem<NS>;
    constexpr uint32_t kIdS = idesc_f16(128, NS, 1, 0, 0);    // with a state's transpose: K-major
    constexpr uint32_t kIdDb = idesc_f16(128, NS, 1, 0, 1), kIdDc = idesc_f16(128, NS, 1, 1, 1);
    const uint32_t base = smem_u32(smem);
    __shared__ uint32_t s_tmem, s_abort;
    Ctx x;
    x.bars = base + L::kBars;
    x.abort = &s_abort;
    x.error = &g_scan_tc_bwd_error;
    HeadGates *gates = reinterpret_cast<HeadGates *>(smem + L::kGates);
    Partials &sums = *reinterpret_cast<Partials *>(smem + L::kSums);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int split_i = static_cast<int>(blockIdx.x % w.splits);
    const int grp = static_cast<int>(blockIdx.x / w.splits % p.G);
    const int64_t unit = blockIdx.x / w.splits / p.G;
    const int per_group = p.H / p.G, per = (per_group + w.splits - 1) / w.splits;
    const int hb = grp * per_group + split_i * per, he = min(hb + per, (grp + 1) * per_group);
    const Piece u = find_piece(p.seqs, unit, TT);
    const int cnt = u.none ? 0 : static_cast<int>(u.b - u.a);
    if (cnt == 0) {
        for (int j = tid; j < 3 * (he - hb); j += NT) w.part[(unit * 3 + j / (he - hb)) * p.H + hb + j % (he - hb)] = 0.f;
        return;
    }
    const int slices = p.P / PC, work = (he - hb) * slices;
    if (work <= 0) return;
    const int64_t start = u.a;

    if (warp == kIssuer) {
        if (lane == 0) {
            for (int i = 0; i < kBarCount; ++i) mbar_init(x.bar(i), i < kByAll ? 1 : i < kQRead ? 16 : 4);
            s_abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp < kIssuer) {
        // ---------------------------------------------------------------- the elements
        // thread: row r (token or state entry, TMEM lane); cq: 32 tokens t, or 16 of a head's columns
        const int wq = warp & 3, cq = warp >> 2, r = wq * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tQ = tmem + kColQ + 32 * cq + lanes, tM = tmem + kColM + 16 * cq + lanes;
        const uint32_t tX = tmem + kColX + 16 * cq + lanes, tY = tmem + kColY + 16 * cq + lanes;
        bool ok = x.met(x.wait(kBcFull, 0));
        if (ok) {
            // rows behind the piece: of other tokens, or none
            uint8_t *t = smem + (cq >> 1 ? L::kB : L::kC) + r * 128 + (NS == 128 ? (cq & 1) * kBlock : (cq & 1) * 64);
            if (r >= cnt)
#pragma unroll
                for (int j = 0; j < NS / 16; ++j) sts(t + j * 16, make_uint4(0u, 0u, 0u, 0u));
            fence_proxy_async_smem();
            x.arrive(kSParts);
        }
        // the same of x and dy, and leave to compute Qt
        auto ready = [&](int k) {
            if (cnt < TT) {
                if (!x.met(x.wait(kXFull + (k & 1), (k >> 1) & 1))) return false;
                uint8_t *t = smem + L::kXY + ((k & 1) * 2 + (cq >> 1)) * kBlock + r * 128 + (cq & 1) * 64;
                if (r >= cnt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sts(t + j * 16, make_uint4(0u, 0u, 0u, 0u));
                fence_proxy_async_smem();
            }
            tc_fence_before();
            x.arrive(kQReady);
            return true;
        };
        // this thread's part of a state matrix: of row sr JS times 8 columns, from 8 (s8 + j) on
        constexpr int JS = NS / 64;
        const int sr = NS == 128 ? r : r & 63, s8 = NS == 128 ? 2 * cq : 2 * cq + (wq >> 1);
        auto state_at = [&](uint32_t tile, int j, int i) {
            if constexpr (NS == 128)
                return *reinterpret_cast<const float4 *>(smem + tile + (cq >> 1) * L::kPart + sw128(r, (cq & 1) * 4 + 2 * j + i));
            else
                return *reinterpret_cast<const float4 *>(smem + tile + (s8 >> 2) * L::kPart + sw128(sr, (s8 & 3) * 2 + i));
        };
        auto part_at = [&](int e, int j) {
            return smem + L::kParts + e * L::kPart + (NS == 128 ? sw128(r, 2 * cq + j) : sw128(sr, s8));
        };
        auto split8 = [&](const float4 &f0, const float4 &f1, uint4 (&o)[3]) {
            uint32_t v[4][3];
            split<3>(f0.x, f0.y, v[0]);
            split<3>(f0.z, f0.w, v[1]);
            split<3>(f1.x, f1.y, v[2]);
            split<3>(f1.z, f1.w, v[3]);
#pragma unroll
            for (int e = 0; e < 3; ++e) o[e] = make_uint4(v[0][e], v[1][e], v[2][e], v[3][e]);
        };
        // the dot of a row of Y or Z, 16 columns, with dy or x
        auto dot_row = [&](const uint32_t (&a)[16], const uint8_t *tile) {
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 v = lds(tile + sw128(r, 2 * cq + j));
                const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s = fma2(make_float2(f32(a[8 * j + 2 * e]), f32(a[8 * j + 2 * e + 1])),
                             make_float2(bf_low(in[e]), bf_high(in[e])), s);
            }
            return s.x + s.y;
        };
        auto add_to = [](float &dst, float v, bool more) { dst = more ? dst + v : v; };
        float2 gt[16];   // Gt, columns 32 cq .. + 32
        ok = ok && x.met(x.wait(kQ, 0));
        if (ok) {
            tc_fence_after();
            uint32_t a[32];
            tmem_ld32(tQ, a);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) gt[j] = make_float2(f32(a[2 * j]), f32(a[2 * j + 1]));
            ok = ready(0);
        }
        for (int k = 0; k < work && ok; ++k) {
            const int hh = k / slices, sl = k % slices, h = hb + hh, stage = k & 1;
            const uint32_t ph = k & 1;
            const HeadGates &g = gates[hh & 1];
            uint8_t *xt = smem + L::kXY + stage * 2 * kBlock, *dyt = xt + kBlock;
            ok = x.met(x.wait(kXFull + stage, (k >> 1) & 1) && x.wait(kGatesFull + (hh & 1), (hh >> 1) & 1) &&
                       (k == 0 || x.wait(kEnd, ph ^ 1)));
            if (!ok) break;
            tc_fence_after();
            // e^Gamma dy and d e^(Gamma_end - Gamma) x: the first operands with S_0^T and R^T, 32 columns for this thread
            {
                const uint8_t *t = cq >> 1 ? xt : dyt;
                const float wt = cq >> 1 ? g.weight[r] : g.from[r];
                const float2 w2 = make_float2(wt, wt);
                uint32_t o[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 v = lds(t + sw128(r, (cq & 1) * 4 + j));
                    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 m = mul2(make_float2(bf_low(in[e]), bf_high(in[e])), w2);
                        o[4 * j + e] = bf_pair(m.x, m.y);
                    }
                }
                tmem_st16(tmem + (cq >> 1 ? kColSx : kColDy) + 16 * (cq & 1) + lanes, o);
            }
            // S_0 in parts
            ok = x.met(x.wait(kSFull, ph));
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < JS; ++j) {
                uint4 o[3];
                split8(state_at(L::kK, j, 0), state_at(L::kK, j, 1), o);
#pragma unroll
                for (int e = 0; e < 3; ++e) sts(part_at(e, j), o[e]);
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            x.arrive(kSParts);
            // ---- Mt, Kt (where S_0 was) and the sums of Mt . Qt
            ok = x.met(x.wait(kSParts, ph ^ 1) && x.wait(kQ, ph ^ 1) && (k == 0 || sl > 0 || x.wait(kSumsFree, (hh - 1) & 1)));
            if (!ok) break;
            tc_fence_after();
            uint32_t m_out[16];
            auto k_at = [&](int j) { return smem + L::kK + (cq >> 1) * kBlock + sw128(r, (cq & 1) * 4 + j); };
            // kind 0: t > s throughout; 1: the diagonal block; 2: that, where it spans more than 2^60
            auto block = [&](auto kind) {
                constexpr int kKind = decltype(kind)::value;
                const float gh = g.hi[r], gl = g.lo[r], ds = g.d[r];
                const float rf = ex2((g.open_hi[cq] - gh) + (g.open_lo[cq] - gl));
                const float2 rf2 = make_float2(rf, rf), ds2 = make_float2(ds, ds);
                float2 col = make_float2(0.f, 0.f), near = make_float2(0.f, 0.f);
                float on_diag = 0.f, q_diag = 0.f;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t a[16];
                    tmem_ld16(tQ + 16 * q, a);
                    float wsum[16];
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t k_out[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = 16 * q + 8 * j + 2 * i;   // t = 32 cq + c and the next
                            const float2 qv = make_float2(f32(a[8 * j + 2 * i]), f32(a[8 * j + 2 * i + 1]));
                            float2 l;
                            if constexpr (kKind == 2) {
                                const float2 th = *reinterpret_cast<const float2 *>(g.hi + 32 * cq + c);
                                const float2 tl = *reinterpret_cast<const float2 *>(g.lo + 32 * cq + c);
                                l = make_float2(ex2((th.x - gh) + (tl.x - gl)), ex2((th.y - gh) + (tl.y - gl)));
                            } else {
                                l = mul2(*reinterpret_cast<const float2 *>(g.col + 32 * cq + c), rf2);
                            }
                            float2 m = mul2(gt[c >> 1], l);
                            const float2 qd = mul2(qv, ds2);
                            float2 kk = mul2(qd, l), hw = mul2(m, qd);
                            if constexpr (kKind == 0) {
                                col = fma2(m, qv, col);
                            } else {
                                // selected, not multiplied: below the diagonal is what other tokens hold
                                const float2 hq = mul2(m, qv);
                                on_diag = c == lane ? hq.x : c + 1 == lane ? hq.y : on_diag;
                                q_diag = c == lane ? qv.x : c + 1 == lane ? qv.y : q_diag;
                                col.x += c > lane ? hq.x : 0.f;
                                col.y += c + 1 > lane ? hq.y : 0.f;
                                hw = make_float2(c > lane ? hw.x : 0.f, c + 1 > lane ? hw.y : 0.f);
                                near.x += hw.x;
                                near.y += hw.y;
                                m = make_float2(c >= lane ? m.x : 0.f, c + 1 >= lane ? m.y : 0.f);
                                kk = make_float2(c >= lane ? kk.x : 0.f, c + 1 >= lane ? kk.y : 0.f);
                            }
                            wsum[8 * j + 2 * i] = hw.x;
                            wsum[8 * j + 2 * i + 1] = hw.y;
                            m_out[c >> 1] = bf_pair(m.x, m.y);
                            k_out[i] = bf_pair(kk.x, kk.y);
                        }
                        sts(k_at(2 * q + j), make_uint4(k_out[0], k_out[1], k_out[2], k_out[3]));
                    }
                    const float row = sum_lanes16(wsum);
                    if (lane < 16) add_to(sums.row[wq][32 * cq + 16 * q + lane], row, sl > 0);
                }
                add_to(sums.col[cq][r], col.x + col.y, sl > 0);
                if constexpr (kKind > 0) {
                    add_to(sums.near[r], near.x + near.y, sl > 0);
                    add_to(sums.diag[r], on_diag, sl > 0);
                    add_to(sums.q[r], q_diag, sl > 0);
                }
            };
            if (cq < wq) {
#pragma unroll
                for (int j = 0; j < 16; ++j) m_out[j] = 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) sts(k_at(j), make_uint4(0u, 0u, 0u, 0u));
            } else if (cq > wq) {
                block(std::integral_constant<int, 0>());
            } else if (!((g.steep >> cq) & 1u)) {
                block(std::integral_constant<int, 1>());
            } else {
                block(std::integral_constant<int, 2>());
            }
            // Mt lies where the four warps of these lanes have read Qt
            tc_fence_before();
            x.arrive(kQRead + wq);
            ok = x.met(x.wait(kQRead + wq, ph));
            if (!ok) break;
            tc_fence_after();
            tmem_st16(tM, m_out);
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            x.arrive(kMk);
            // ---- the dots with C S_0; R in parts where S_0's were, and the two's product
            ok = x.met(x.wait(kSDone, ph));
            if (!ok) break;
            tc_fence_after();
            {
                uint32_t a[16];
                tmem_ld16(tY, a);
                tmem_wait_ld();
                add_to(sums.leave[cq][r], dot_row(a, dyt), sl > 0);
            }
            ok = x.met(x.wait(kRFull, ph));
            if (!ok) break;
            float2 rs2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < JS; ++j) {
                uint4 o[3];
                const float4 f0 = state_at(L::kXY + (stage ^ 1) * 2 * kBlock, j, 0);
                const float4 f1 = state_at(L::kXY + (stage ^ 1) * 2 * kBlock, j, 1);
                const float2 f[4] = {make_float2(f0.x, f0.y), make_float2(f0.z, f0.w), make_float2(f1.x, f1.y), make_float2(f1.z, f1.w)};
#pragma unroll
                for (int e = 2; e >= 0; --e) {
                    const uint4 v = lds(part_at(e, j));
                    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) rs2 = fma2(f[i], make_float2(bf_low(in[i]), bf_high(in[i])), rs2);
                }
                split8(f0, f1, o);
#pragma unroll
                for (int e = 0; e < 3; ++e) sts(part_at(e, j), o[e]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            x.arrive(kRParts);
            {
                float rs = rs2.x + rs2.y;
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, m);
                if (lane == 0) add_to(sums.rs[warp], rs, sl > 0);
            }
            // ---- dx, and the dots with B R
            ok = x.met(x.wait(kZ, ph));
            if (!ok) break;
            tc_fence_after();
            {
                uint32_t a[16], b[16];
                tmem_ld16(tY, a);
                tmem_ld16(tX, b);
                tmem_wait_ld();
                if (k + 1 < work) {
                    ok = ready(k + 1);
                    if (!ok) break;
                }
                add_to(sums.enter[cq][r], dot_row(a, xt), sl > 0);
                if (r < cnt) {
                    const float d = g.d[r], wt = g.weight[r], Dh = g.D;
                    const float2 d2 = make_float2(d, d), wt2 = make_float2(wt, wt), D2 = make_float2(Dh, Dh);
                    uint16_t *dst = p.dx + (start + r) * p.dx_stride + static_cast<int64_t>(h) * p.P + sl * PC + 16 * cq;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 v = lds(dyt + sw128(r, 2 * cq + j));
                        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = 8 * j + 2 * e;
                            const float2 y = fma2(wt2, make_float2(f32(a[c]), f32(a[c + 1])),
                                                  mul2(D2, make_float2(bf_low(in[e]), bf_high(in[e]))));
                            const float2 z = fma2(d2, make_float2(f32(b[c]), f32(b[c + 1])), y);
                            o[e] = bf_pair(z.x, z.y);
                        }
                        *reinterpret_cast<uint4 *>(dst + 8 * j) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
            if (sl == slices - 1) x.arrive(kSums);
        }
        ok = ok && x.met(x.wait(kEnd, (work - 1) & 1));
        tc_fence_after();
        // ---- dB and dC: this CTA's share, or the result where it has the whole group
        if (ok) {
#pragma unroll
            for (int i = 0; i < NS / 64; ++i) {
                // 0: dB, 1: dC; 32 columns for this thread
                const int which = NS == 128 ? i : cq >> 1, c32 = NS == 128 ? cq : cq & 1;
                uint32_t a[32];
                tmem_ld32(tmem + (which ? kColDc : kColDb) + 32 * c32 + lanes, a);
                tmem_wait_ld();
                const int64_t at_n = static_cast<int64_t>(grp) * NS + 32 * c32;
                if (r >= cnt) continue;
                if (w.dbc) {
                    // planes: the splits' dB, then their dC
                    float *d = w.dbc + (split_i + (which ? w.splits : 0)) * (p.rows * p.G * NS) + (start + r) * p.G * NS + at_n;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        reinterpret_cast<float4 *>(d)[j] =
                            make_float4(f32(a[4 * j]), f32(a[4 * j + 1]), f32(a[4 * j + 2]), f32(a[4 * j + 3]));
                } else {
                    uint16_t *d = (which ? p.dC + (start + r) * p.dc_stride : p.dB + (start + r) * p.db_stride) + at_n;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        reinterpret_cast<uint4 *>(d)[j] =
                            make_uint4(bf_pair(f32(a[8 * j]), f32(a[8 * j + 1])), bf_pair(f32(a[8 * j + 2]), f32(a[8 * j + 3])),
                                       bf_pair(f32(a[8 * j + 4]), f32(a[8 * j + 5])), bf_pair(f32(a[8 * j + 6]), f32(a[8 * j + 7])));
                }
            }
        }
    } else if (warp == kIssuer) {
        // ---------------------------------------------------------------- loads and products
        auto load_xy = [&](int k) {
            if (elect_one()) {
                const int stage = k & 1;
                const int32_t col = (hb + k / slices) * p.P + (k % slices) * PC, row = static_cast<int32_t>(start);
                const uint32_t d = base + L::kXY + stage * 2 * kBlock;
                mbar_arrive_expect_tx(x.bar(kXFull + stage), 2 * kBlock);
                tma_load_2d(d, &maps.x, x.bar(kXFull + stage), col, row);
                tma_load_2d(d + kBlock, &maps.dy, x.bar(kXFull + stage), col, row);
            }
            __syncwarp();
        };
        const uint32_t bt = base + L::kB, ct = base + L::kC, parts = base + L::kParts, kt = base + L::kK;
        auto k_major = [&](uint32_t tile, int k) {   // step k of 16 columns
            return smem_desc(tile + (k >> 2) * kBlock + (k & 3) * 32, 16, 1024, kSwizzle128);
        };
        auto mn_major = [&](uint32_t tile, int k) {  // step k of 16 rows
            return smem_desc(tile + k * 2048, kBlock, 1024, kSwizzle128);
        };
        // fp32 states, two blocks of 32 columns
        auto load_state = [&](int k, const CUtensorMap *map, int bar, uint32_t dst) {
            if (elect_one()) {
                const int32_t row = static_cast<int32_t>((unit * p.H + hb + k / slices) * NS), col = (k % slices) * PC;
                mbar_arrive_expect_tx(x.bar(bar), 2 * L::kPart);
                for (int j = 0; j < 2; ++j) tma_load_2d(base + dst + j * L::kPart, map, x.bar(bar), col + 32 * j, row);
            }
            __syncwarp();
        };
        if (elect_one()) {
            mbar_arrive_expect_tx(x.bar(kBcFull), 2 * L::kTile);
            for (int k = 0; k < NS / 64; ++k) {
                tma_load_2d(ct + k * kBlock, &maps.c, x.bar(kBcFull), grp * NS + 64 * k, static_cast<int32_t>(start));
                tma_load_2d(bt + k * kBlock, &maps.b, x.bar(kBcFull), grp * NS + 64 * k, static_cast<int32_t>(start));
            }
        }
        __syncwarp();
        load_xy(0);
        load_state(0, &maps.states, kSFull, L::kK);
        bool ok = x.met(x.wait(kBcFull, 0) && x.wait(kSParts, 0));
        if (ok) {
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < NS / 16; ++k) mma_f16(tmem + kColQ, k_major(bt, k), k_major(ct, k), kIdQ, k > 0);
                mma_commit(x.bar(kQ));
            }
            __syncwarp();
        }
        for (int k = 0; k < work && ok; ++k) {
            const int stage = k & 1;
            const uint32_t ph = k & 1, xt = base + L::kXY + stage * 2 * kBlock, dyt = xt + kBlock;
            ok = x.met(x.wait(kXFull + stage, (k >> 1) & 1) && x.wait(kQReady, ph));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_f16(tmem + kColQ, k_major(xt, j), k_major(dyt, j), kIdQ, j > 0);
                mma_commit(x.bar(kQ));
            }
            __syncwarp();
            ok = x.met(x.wait(kSParts, ph ^ 1));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < NS / 16; ++j)
#pragma unroll
                    for (int e = 2; e >= 0; --e)
                        mma_f16(tmem + kColY, k_major(ct, j), mn_major(parts + e * L::kPart, j), kIdY, !(j == 0 && e == 2));
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 1; e >= 0; --e)
                        mma_f16_ts(tmem + kColDc, tmem + kColDy + 8 * j, k_major(parts + e * L::kPart, j), kIdS,
                                   !(k == 0 && j == 0 && e == 1));
                mma_commit(x.bar(kSDone));
            }
            __syncwarp();
            load_state(k, &maps.grads, kRFull, L::kXY + (stage ^ 1) * 2 * kBlock);
            ok = x.met(x.wait(kMk, ph));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    mma_f16_ts(tmem + kColX, tmem + kColM + 8 * j, mn_major(dyt, j), kIdY, j > 0);
#pragma unroll
                for (int j = 0; j < 8; ++j) mma_f16(tmem + kColDc, mn_major(kt, j), mn_major(bt, j), kIdDc, 1);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    mma_f16(tmem + kColDb, k_major(kt, j), mn_major(ct, j), kIdDb, !(k == 0 && j == 0));
            }
            __syncwarp();
            ok = x.met(x.wait(kRParts, ph));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < NS / 16; ++j)
#pragma unroll
                    for (int e = 2; e >= 0; --e)
                        mma_f16(tmem + kColY, k_major(bt, j), mn_major(parts + e * L::kPart, j), kIdY, !(j == 0 && e == 2));
                mma_commit(x.bar(kZ));
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 1; e >= 0; --e)
                        mma_f16_ts(tmem + kColDb, tmem + kColSx + 8 * j, k_major(parts + e * L::kPart, j), kIdS, 1);
                mma_commit(x.bar(kEnd));
            }
            __syncwarp();
            if (k + 1 < work) {
                load_xy(k + 1);
                ok = x.met(x.wait(kEnd, ph));   // Kt has been multiplied
                if (!ok) break;
                load_state(k + 1, &maps.states, kSFull, L::kK);
            }
        }
    } else {
        // ---------------------------------------------------------------- gates a head ahead, and the last head's sums
        const int t4 = 4 * lane;
        float dt[4], A = 0.f, bias = 0.f, D = 0.f;
        auto fetch = [&](int h) {
#pragma unroll
            for (int j = 0; j < 4; ++j) dt[j] = t4 + j < cnt ? p.dt[(start + t4 + j) * p.H + h] : 0.f;
            A = p.A[h];
            bias = p.dt_bias ? p.dt_bias[h] : 0.f;
            D = p.D ? p.D[h] : 0.f;
        };
        const int heads = he - hb;
        bool ok = true;
        fetch(hb);
        for (int hh = 0; hh < heads + 1 && ok; ++hh) {
            if (hh < heads) {
                make_head_gates(gates[hh & 1], dt, cnt, A, bias, D, p.softplus);
#ifdef KDA_TEST_HOOKS
                if (hh != g_scan_tc_bwd_stall)
#endif
                x.arrive(kGatesFull + (hh & 1));
                if (hh + 1 < heads) {
                    fetch(hb + hh + 1);
                }
            }
            if (hh == 0) continue;
            // the head before: its gates, and then the place of the next one's
            const int h = hb + hh - 1;
            const HeadGates &g = gates[(hh - 1) & 1];
            ok = x.met(x.wait(kSums, (hh - 1) & 1));
            if (!ok) break;
            // Pairs s < t <= u of dlog a_t: within t's quarter they are what its later rows have more than its later
            // columns, and only there is anything subtracted; with one of the two or both in other quarters they are sums.
            float own[4], to_u[4], from_s[4], lv[4], in[4], dd[4], qq[4], z1 = 0.f, z2 = 0.f;
            const int quarter = lane >> 3;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t4 + j;
                float l = 0.f, en = 0.f, row = 0.f, col = 0.f, c0 = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l += sums.leave[e][t];
                    en += sums.enter[e][t];
                    if (e < quarter) row += sums.row[e][t];
                    if (e > quarter) col += sums.col[e][t];
                    if (e == quarter) {
                        own[j] = sums.row[e][t] - sums.near[t];
                        c0 = sums.col[e][t];
                    }
                }
                if (quarter >= 2) z1 += sums.row[0][t];
                if (quarter == 3) z2 += sums.row[0][t] + sums.row[1][t];
                en *= g.to[t];
                to_u[j] = row;
                from_s[j] = g.d[t] * col;
                lv[j] = g.from[t] * l;
                in[j] = g.d[t] * en;
                dd[j] = c0 + col + sums.diag[t] + en;
                qq[j] = sums.q[t];
            }
            float rs = lane < 16 ? sums.rs[lane] : 0.f;
            x.arrive(kSumsFree);
#pragma unroll
            for (int m = 8; m > 0; m >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, m);
            rs = g.total * __shfl_sync(0xffffffffu, rs, 0);
            // sums over later (earlier) tokens: over the tile, and over the quarter
            float later = (lv[0] + lv[1]) + (lv[2] + lv[3]), earlier = (in[0] + in[1]) + (in[2] + in[3]);
            float later8 = (own[0] + own[1]) + (own[2] + own[3]), cross8 = (to_u[0] + to_u[1]) + (to_u[2] + to_u[3]);
            float earlier8 = (from_s[0] + from_s[1]) + (from_s[2] + from_s[3]);
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const float a = __shfl_down_sync(0xffffffffu, later, m), b = __shfl_up_sync(0xffffffffu, earlier, m);
                if (lane + m < 32) later += a;
                if (lane >= m) earlier += b;
                z1 += __shfl_xor_sync(0xffffffffu, z1, m);
                z2 += __shfl_xor_sync(0xffffffffu, z2, m);
                if (m < 8) {
                    const float c = __shfl_down_sync(0xffffffffu, later8, m), d = __shfl_down_sync(0xffffffffu, cross8, m);
                    const float e = __shfl_up_sync(0xffffffffu, earlier8, m);
                    if ((lane & 7) + m < 8) {
                        later8 += c;
                        cross8 += d;
                    }
                    if ((lane & 7) >= m) earlier8 += e;
                }
            }
            auto before_lane = [&](float v, int width) {
                const float o = __shfl_up_sync(0xffffffffu, v, 1);
                return lane & (width - 1) ? o : 0.f;
            };
            auto behind_lane = [&](float v, int width) {
                const float o = __shfl_down_sync(0xffffffffu, v, 1);
                return (lane & (width - 1)) < width - 1 ? o : 0.f;
            };
            later = behind_lane(later, 32);
            later8 = behind_lane(later8, 8);
            cross8 = behind_lane(cross8, 8);
            earlier = before_lane(earlier, 32);
            earlier8 = before_lane(earlier8, 8);
            const float far = rs + (quarter == 1 ? z1 : quarter == 2 ? z2 : 0.f);
            float dl[4];
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                later += lv[j];
                later8 += own[j];
                cross8 += to_u[j];
                dl[j] = (later8 + cross8) + (later + far);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dl[j] += earlier + earlier8;
                earlier += in[j];
                earlier8 += from_s[j];
            }
            float sa = 0.f, sb = 0.f, sd = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t4 + j;
                if (t < cnt) {
                    const float v = fmaf(dl[j], g.A, dd[j]) * g.slope[t];
                    p.ddt[(start + t) * p.H + h] = v;
                    sa = fmaf(dl[j], g.d[t], sa);
                    sb += v;
                    sd += qq[j];
                }
            }
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) {
                sa += __shfl_xor_sync(0xffffffffu, sa, m);
                sb += __shfl_xor_sync(0xffffffffu, sb, m);
                sd += __shfl_xor_sync(0xffffffffu, sd, m);
            }
            if (lane == 0) {
                w.part[(unit * 3 + 0) * p.H + h] = sa;
                w.part[(unit * 3 + 1) * p.H + h] = sb;
                w.part[(unit * 3 + 2) * p.H + h] = sd;
            }
            __syncwarp();
        }
    }
    if (s_abort) {
        // copies may still be in flight into this CTA's shared memory
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 20000000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

}  // namespace tc
}  // namespace scan

namespace scan {
namespace tc {

template <int NS>
cudaError_t bwd_launch(const ScanParams &p, const BwdWork &w, cudaStream_t s) {
    const int64_t ctas = w.cells * p.G * w.splits;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    BwdMaps maps;
    memset(&maps, 0, sizeof(maps));
    const int64_t hp = static_cast<int64_t>(p.H) * p.P, gn = static_cast<int64_t>(p.G) * NS, all = w.cells * p.H * NS;
    constexpr auto type = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    if (p.rows > 0 && (!encode(&maps.states, type, 4, w.states, p.P, all, p.P, NS) ||
                       !encode(&maps.grads, type, 4, w.grads, p.P, all, p.P, NS) ||
                       !encode(&maps.x, p.x, hp, p.rows, p.x_stride, TT) ||
                       !encode(&maps.dy, p.dout, hp, p.rows, p.dout_stride, TT) ||
                       !encode(&maps.b, p.B, gn, p.rows, p.b_stride, TT) || !encode(&maps.c, p.C, gn, p.rows, p.c_stride, TT)))
        return cudaErrorInvalidValue;
    cudaError_t err = allow_smem(scan_tc_bwd_kernel<NS>, BwdSmem<NS>::kBytes);
    if (err != cudaSuccess) return err;
    scan_tc_bwd_kernel<NS><<<static_cast<unsigned>(ctas), NT, BwdSmem<NS>::kBytes, s>>>(p, w, maps);
    return cudaGetLastError();
}

}  // namespace tc
}  // namespace scan

cudaError_t launch_scan_tc_bwd(const ScanParams &p, const BwdWork &w, cudaStream_t s) {
    return p.N == 128 ? scan::tc::bwd_launch<128>(p, w, s) : scan::tc::bwd_launch<64>(p, w, s);
}

cudaError_t read_and_clear_scan_tc_bwd_error(unsigned int *value) {
    cudaError_t err = cudaMemcpyFromSymbol(value, scan::tc::g_scan_tc_bwd_error, sizeof(*value));
    if (err != cudaSuccess || *value == 0) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(scan::tc::g_scan_tc_bwd_error, &zero, sizeof(zero));
}

#ifdef KDA_TEST_HOOKS
extern "C" int kda_test_set_scan_tc_bwd_stall(int at) {
    return static_cast<int>(cudaMemcpyToSymbol(scan::tc::g_scan_tc_bwd_stall, &at, sizeof(int)));
}
#endif

}  // namespace kda
