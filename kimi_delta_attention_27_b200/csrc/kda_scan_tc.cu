// kda_scan_tc.cu -- selective state space scan over prompts on tcgen05, state size 128, sm_100a.
//
// The recurrence and its tile form are those of kda_scan_fwd.cu, with tiles of 128 tokens: 128 is the M of a
// tcgen05 product and the number of TMEM lanes, so that C B^T, y and the state (rows: its 128 entries) each have
// one row per lane and one thread per row. Per tile and 64 columns of a head:
//
//   G  = C B^T                              128 x 128, K 128     once for both heads of the CTA
//   Y1 = C S_0 (bf16 copy of the state)     128 x 64,  K 128     y = e^Gamma Y1 + Y2 + D x
//   Y2 = (L . G d) x                        128 x 64,  K 128     the first operand from TMEM, in bf16
//   U  = B^T (d e^(Gamma_end - Gamma) x)    128 x 64,  K 128     the second operand in 2 or 3 bf16 parts
//   S  = e^(Gamma_end) S_0 + U                                   fp32, in the registers of 256 threads
//
// What bounds it: for two heads' tile the products take 2600 cycles, the elements' traffic with shared memory and TMEM
// 4100, their instructions (L . G, the parts of x, scaling and rounding) 3900 of each scheduler, HBM 3000 (68 KB); what is
// left is the chain from one tile's state to the next. So eight warps take each of two heads (of the same group, so that
// they share C, B and G, and one product with N = 128 reads C or B^T once for both), a thread having half of a row; one
// thread issues the products; two warps run ahead with the gates and the loads of x. A tile's outputs are finished in the
// next tile, between the two halves of its parts, so that no product is waited for while there is work, and nothing but
// Y1 waits for the state. (65536 tokens x 32 heads x 128 in pieces: 553 us, 9700 cycles for two heads' tile; with Y1 and U
// by head 584; warp-level products with tiles of 64 tokens 1.13 ms.)
//
// L . G is formed without one exponential per element: with a_b = Gamma at the end of a block of 32 columns,
// L_ts = e^(Gamma_t - a_b) e^(a_b - Gamma_s), a factor per row and one per column, both at most 1 for the
// rows behind the block. In the block on the diagonal the row's factor is above 1; where the sums lie more than 2^60 from
// the block's end (they may on either side: a negative step lets the state grow) its elements take an exponential each
// instead.
//
// Every wait is bounded; one that runs out raises kErrTimeout and winds the CTA down.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_scan_tc.cuh"

namespace kda {
namespace scan {
namespace tc {

__device__ unsigned int g_scan_tc_error = 0;
#ifdef KDA_TEST_HOOKS
// Test-only build (never the product library): the gates of this tile of every CTA are not signalled, so that the bounded
// waits for them run out.
__device__ int g_scan_tc_stall = -1;
#endif

constexpr int TT = kScanTcTile;           // tokens per tile
constexpr int NT = 608;                   // eight warps for each head, an issuing warp, two for the gates
constexpr int kIssuer = 16, kFeeder = 17; // the others' first warps

struct TcGates {
    float hi[TT], lo[TT];   // log2 of the decay from the tile's start through token t, in two floats
    float d[TT];            // the steps
    float col[TT];          // d e^(a_b - Gamma): the column factors of L . G d
    float from[TT];         // e^Gamma
    float weight[TT];       // d e^(Gamma_end - Gamma)
    float total;
    uint32_t steep;         // bit b: the decays within block b of 32 span more than 2^60
    float pad[2];
};

template <int S>
struct Smem {
    static constexpr uint32_t kC = 0, kB = 2 * kBlock, kX = 4 * kBlock;    // x: [head][stage]
    static constexpr uint32_t kState = kX + 4 * kBlock;                    // [head]: the state in bf16
    static constexpr uint32_t kPart = 64 * 128;                            // 64 tokens of one part
    static constexpr uint32_t kParts = kState + 2 * kBlock;                // [S][head]
    static constexpr uint32_t kGates = kParts + 2 * S * kPart;             // [head][stage]
    static constexpr uint32_t kBars = kGates + 4 * sizeof(TcGates);
    static constexpr uint32_t kBytes = kBars + 512;
    static_assert(kBytes <= 227 * 1024, "shared memory of one CTA");
};

// TMEM columns: G, then both heads' U, Y1 and Y2. M (L . G d in bf16 pairs) takes U's place once that has been read.
constexpr uint32_t kColG = 0, kColU = 128, kColY1 = 256, kColY2 = 384, kColHead = 64, kCols = 512;

constexpr uint32_t kIdG = idesc_f16(128, 128, 1, 0, 0);   // C and B, both K-major
constexpr uint32_t kIdY = idesc_f16(128, 64, 1, 0, 1);    // M K-major, x MN-major

struct Maps {
    CUtensorMap x, b, c;
};

// barriers, 8 bytes each behind Smem::kBars
enum : int {
    kBcFull = 0,        // C and B of a tile
    kG = 2,             // G is there
    kXFull = 3,         // [head][stage] x
    kGates = 7,         // [head][stage] the gates
    kPFree = 11,        // the first half's product is done
    kU = 12,            // U is there
    kY = 13,            // [head] Y1 and Y2 are there
    kByHead = 15,       // from here on: the head's eight warps arrive
    kXFree = 15,        // [head][stage] the tile's x and gates have been used
    kS = 19,            // [head] the state's copy is written
    kYFree = 21,        // [head] Y1 and Y2 have been read
    kP0 = 23, kP1 = 25, // [head] the parts of the tile's first, second 64 tokens are written
    kM = 27,            // [head] M is written
    kBarCount = 29
};

// the steps of a lane's tokens 4l .. 4l + 3 before bias and softplus (0 behind the tile)
__device__ __forceinline__ void load_dt(const ScanParams &p, int64_t start, int cnt, int h, float (&dt)[4]) {
    const int t = 4 * (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < 4; ++j) dt[j] = t + j < cnt ? p.dt[(start + t + j) * p.H + h] : 0.f;
}

// The gates of a tile of cnt tokens, by one warp: lane l has tokens 4l .. 4l + 3.
__device__ __forceinline__ void make_tc_gates(TcGates &g, const float (&dt)[4], int cnt, float bias, int softplus, Two a2) {
    const int lane = threadIdx.x & 31;
    float d[4];
    Two c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float u;
        d[j] = 4 * lane + j < cnt ? step_of(dt[j], bias, softplus, &u) : 0.f;
        c[j] = 4 * lane + j < cnt ? log_decay(d[j], a2) : Two{0.f, 0.f};
        if (j) c[j] = c[j - 1] + c[j];
    }
    const Two s = scan_lanes(c[3]), total = shfl(s, 31);
    Two before = {__shfl_up_sync(0xffffffffu, s.hi, 1), __shfl_up_sync(0xffffffffu, s.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const Two anchor = shfl(s, lane | 7), opens = shfl(before, lane & 24);   // the block's end and start
    float hi[4], lo[4], col[4], from[4], weight[4];
    const float whole = minus(opens, anchor);
    float span = fabsf(whole);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const Two v = before + c[j];
        hi[j] = v.hi;
        lo[j] = v.lo;
        const float to_end = minus(anchor, v);
        span = fmaxf(span, fabsf(to_end));
        col[j] = d[j] * ex2(to_end);
        from[j] = ex2(v);
        weight[j] = d[j] * ex2(minus(total, v));
    }
    // by eight lanes of a block each; a NaN counts, for it must not reach the tokens before it
    const unsigned steep = __ballot_sync(0xffffffffu, span > 60.f || isnan(whole));
    reinterpret_cast<float4 *>(g.hi)[lane] = make_float4(hi[0], hi[1], hi[2], hi[3]);
    reinterpret_cast<float4 *>(g.lo)[lane] = make_float4(lo[0], lo[1], lo[2], lo[3]);
    reinterpret_cast<float4 *>(g.d)[lane] = make_float4(d[0], d[1], d[2], d[3]);
    reinterpret_cast<float4 *>(g.col)[lane] = make_float4(col[0], col[1], col[2], col[3]);
    reinterpret_cast<float4 *>(g.from)[lane] = make_float4(from[0], from[1], from[2], from[3]);
    reinterpret_cast<float4 *>(g.weight)[lane] = make_float4(weight[0], weight[1], weight[2], weight[3]);
    if (lane == 0) {
        g.total = ex2(total);
        g.steep = steep_blocks(steep);
    }
}

template <int S>
__global__ void __launch_bounds__(NT, 1)
    scan_tc_kernel(ScanParams p, const __grid_constant__ Maps maps, int64_t seg, const float *entering) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = Smem<S>;
    const uint32_t base = smem_u32(smem);
    __shared__ uint32_t s_tmem, s_abort;
    Ctx x;
    x.bars = base + L::kBars;
    x.abort = &s_abort;
    x.error = &g_scan_tc_error;
    TcGates *gates = reinterpret_cast<TcGates *>(smem + L::kGates);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0) check_offsets(p.seqs, &g_scan_tc_error);

    // the CTA's piece and its one or two heads ("heads" here: runs of 64 columns of x, of one group)
    const int slices = p.P / PC, per_group = p.H / p.G * slices, pairs = (per_group + 1) / 2;
    const int64_t unit = blockIdx.x / (p.G * pairs);
    const int gp = static_cast<int>(blockIdx.x % (p.G * pairs)), grp = gp / pairs, in_group = gp % pairs * 2;
    const int v0 = grp * per_group + in_group, heads = in_group + 1 < per_group ? 2 : 1;
    const Piece u = find_piece(p.seqs, unit, seg);
    if (u.none) return;
    const int64_t c_first = u.a / TT;
    const int tiles = static_cast<int>(u.b > u.a ? (u.b + TT - 1) / TT - c_first : 0);
    auto start_of = [&](int i) { return (c_first + i) * TT > u.a ? (c_first + i) * TT : u.a; };
    auto count_of = [&](int i) {
        const int64_t e = (c_first + i + 1) * TT < u.b ? (c_first + i + 1) * TT : u.b;
        return static_cast<int>(e - start_of(i));
    };

    if (warp == kIssuer) {
        if (lane == 0) {
            for (int i = 0; i < kBarCount; ++i) mbar_init(x.bar(i), i < kByHead ? 1 : 8);
            s_abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(smem_u32(&s_tmem), kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp < kIssuer) {
        // ---------------------------------------------------------------- a head's elements
        // thread: row r (token or state entry, TMEM lane) and columns 32 hf .. + 32
        const int hd = warp >> 3, hf = (warp >> 2) & 1, wq = warp & 3, r = wq * 32 + lane, t256 = tid & 255;
        if (hd < heads) {
            const int v = v0 + hd, h = v / slices, col = v % slices * PC + 32 * hf;
            const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
            const uint32_t tU = tmem + kColU + hd * kColHead + 32 * hf + lanes, tG = tmem + kColG + lanes;
            const uint32_t tY1 = tmem + kColY1 + hd * kColHead + 32 * hf + lanes;
            const uint32_t tY2 = tmem + kColY2 + hd * kColHead + 32 * hf + lanes;
            uint8_t *st = smem + L::kState + hd * kBlock, *parts = smem + L::kParts + hd * L::kPart;
            const int64_t sn = static_cast<int64_t>(N) * p.P;
            const float Dh = p.D ? p.D[h] : 0.f;
            float2 s[16];         // this thread's part of the state
            {
                const void *src = entering ? entering : p.h0;
                const bool fp32 = entering || p.h0_fp32;
                const int64_t e = ((entering ? unit : static_cast<int64_t>(u.i)) * p.H + h) * sn +
                                  static_cast<int64_t>(r) * p.P + col;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (src && fp32) {
                        f = reinterpret_cast<const float4 *>(static_cast<const float *>(src) + e)[j];
                    } else if (src) {
                        const uint2 w = reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(src) + e)[j];
                        f = make_float4(bf_low(w.x), bf_high(w.x), bf_low(w.y), bf_high(w.y));
                    }
                    s[2 * j] = make_float2(f.x, f.y);
                    s[2 * j + 1] = make_float2(f.z, f.w);
                }
            }
            auto publish = [&]() {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sts(st + sw128(r, 4 * hf + j),
                        make_uint4(bf_pair(s[4 * j].x, s[4 * j].y), bf_pair(s[4 * j + 1].x, s[4 * j + 1].y),
                                   bf_pair(s[4 * j + 2].x, s[4 * j + 2].y), bf_pair(s[4 * j + 3].x, s[4 * j + 3].y)));
                fence_proxy_async_smem();
                x.arrive(kS + hd);
            };
            // d e^(Gamma_end - Gamma) x of 64 tokens in bf16 parts; four threads per token
            auto write_parts = [&](int half, uint8_t *xt, const TcGates &g, int cnt) {
                const int row = half * 64 + (t256 >> 2);
                const float w = g.weight[row];
                const float2 w2 = make_float2(w, w), minus1 = make_float2(-1.f, -1.f);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int chunk = (t256 & 3) * 2 + j;   // two rows' chunks of a turn lie in different banks
                    uint32_t o[S][4];
                    if (row < cnt) {
                        const uint4 q = lds(xt + sw128(row, chunk));
                        const uint32_t in[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float2 f = mul2(make_float2(bf_low(in[k]), bf_high(in[k])), w2);
#pragma unroll
                            for (int e = 0; e < S; ++e) {
                                o[e][k] = bf_pair(f.x, f.y);
                                if (e + 1 < S) f = fma2(make_float2(bf_low(o[e][k]), bf_high(o[e][k])), minus1, f);
                            }
                        }
                    } else {
                        // rows behind the piece: of other tokens, or none
#pragma unroll
                        for (int e = 0; e < S; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0u;
                        sts(xt + sw128(row, chunk), make_uint4(0u, 0u, 0u, 0u));
                    }
#pragma unroll
                    for (int e = 0; e < S; ++e)
                        sts(parts + e * 2 * L::kPart + sw128(t256 >> 2, chunk), make_uint4(o[e][0], o[e][1], o[e][2], o[e][3]));
                }
                fence_proxy_async_smem();
                x.arrive((half ? kP1 : kP0) + hd);
            };
            // y = e^Gamma Y1 + Y2 + D x of tile i, by way of x's own rows in shared memory
            auto finish = [&](int i) {
                const int stage = i & 1, cnt = count_of(i);
                uint8_t *xt = smem + L::kX + (hd * 2 + stage) * kBlock;
                if (!x.met(x.wait(kY + hd, i & 1))) return false;
                tc_fence_after();
                const float f = gates[hd * 2 + stage].from[r];
                const float2 f2 = make_float2(f, f), D2 = make_float2(Dh, Dh);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t a[16], b[16];
                    tmem_ld16(tY1 + 16 * q, a);
                    tmem_ld16(tY2 + 16 * q, b);
                    tmem_wait_ld();
                    if (q == 1) {
                        tc_fence_before();
                        x.arrive(kYFree + hd);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint8_t *at_x = xt + sw128(r, 4 * hf + 2 * q + j);
                        const uint4 w = lds(at_x);
                        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int e = 8 * j + 2 * k;
                            const float2 y =
                                fma2(make_float2(f32(a[e]), f32(a[e + 1])), f2, make_float2(f32(b[e]), f32(b[e + 1])));
                            const float2 z = fma2(make_float2(bf_low(in[k]), bf_high(in[k])), D2, y);
                            o[k] = bf_pair(z.x, z.y);
                        }
                        sts(at_x, make_uint4(o[0], o[1], o[2], o[3]));
                    }
                }
                // the warp's rows, 64 bytes of each
                __syncwarp();
                const int chunk = 4 * hf + (lane & 3);
                uint16_t *out = p.out + start_of(i) * p.out_stride + static_cast<int64_t>(v) * PC + chunk * 8;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // rows four apart side by side: their chunks lie in different banks
                    const int row = wq * 32 + j * 8 + (lane & 4) + (lane >> 3);
                    if (row < cnt) *reinterpret_cast<uint4 *>(out + row * p.out_stride) = lds(xt + sw128(row, chunk));
                }
                fence_proxy_async_smem();   // x's next load comes after these reads and writes
                x.arrive(kXFree + hd * 2 + stage);
                return true;
            };
            bool ok = true;
            if (tiles > 0) publish();
            for (int i = 0; i < tiles && ok; ++i) {
                const int stage = i & 1, cnt = count_of(i);
                const uint32_t ph = i & 1, ph2 = (i >> 1) & 1;
                uint8_t *xt = smem + L::kX + (hd * 2 + stage) * kBlock;
                const TcGates &g = gates[hd * 2 + stage];
                ok = x.met(x.wait(kXFull + hd * 2 + stage, ph2) && x.wait(kGates + hd * 2 + stage, ph2));
                if (!ok) break;
                if (cnt < TT && hd == 0) {
                    // rows of B behind the piece: whatever they hold would multiply zeros below
                    ok = x.met(x.wait(kBcFull, ph));
                    if (!ok) break;
                    uint8_t *bt = smem + L::kB + hf * kBlock;
                    if (r >= cnt)
#pragma unroll
                        for (int j = 0; j < 8; ++j) sts(bt + r * 128 + j * 16, make_uint4(0u, 0u, 0u, 0u));
                }
                write_parts(0, xt, g, cnt);
                if (i > 0) {
                    ok = finish(i - 1);
                    if (!ok) break;
                }
                ok = x.met(x.wait(kPFree, ph));
                if (!ok) break;
                write_parts(1, xt, g, cnt);
                // S = e^(Gamma_end) S + U
                ok = x.met(x.wait(kU, ph));
                if (!ok) break;
                tc_fence_after();
                {
                    const float2 tot = make_float2(g.total, g.total);
                    uint32_t a[32];
                    tmem_ld32(tU, a);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = fma2(s[j], tot, make_float2(f32(a[2 * j]), f32(a[2 * j + 1])));
                }
                // the state's copy: C S_0 of this tile has been computed, as the product behind it has
                if (i + 1 < tiles) publish();
                // M = L . G d in U's place: rows r, blocks of 32 columns, two for each half
                ok = x.met(x.wait(kG, ph));
                if (!ok) break;
                tc_fence_after();
                const float gh = g.hi[r], glo = g.lo[r];
#pragma unroll
                for (int bb = 0; bb < 2; ++bb) {
                    const int b = 2 * hf + bb;
                    uint32_t o[16];
                    if (b > wq) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = 0u;
                    } else {
                        uint32_t a[32];
                        tmem_ld32(tG + 32 * b, a);
                        const int e = 32 * b + 31;
                        if (b < wq || !((g.steep >> b) & 1u)) {
                            const float rf = ex2((gh - g.hi[e]) + (glo - g.lo[e]));
                            const float2 rf2 = make_float2(rf, rf);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float4 cf = reinterpret_cast<const float4 *>(g.col + 32 * b)[j];
                                const float2 m0 =
                                    mul2(mul2(make_float2(f32(a[4 * j]), f32(a[4 * j + 1])), make_float2(cf.x, cf.y)), rf2);
                                const float2 m1 =
                                    mul2(mul2(make_float2(f32(a[4 * j + 2]), f32(a[4 * j + 3])), make_float2(cf.z, cf.w)), rf2);
                                if (b < wq) {
                                    o[2 * j] = bf_pair(m0.x, m0.y);
                                    o[2 * j + 1] = bf_pair(m1.x, m1.y);
                                } else {
                                    // selected, not multiplied: above the diagonal is what later tokens hold
                                    o[2 * j] = bf_pair(4 * j <= lane ? m0.x : 0.f, 4 * j + 1 <= lane ? m0.y : 0.f);
                                    o[2 * j + 1] = bf_pair(4 * j + 2 <= lane ? m1.x : 0.f, 4 * j + 3 <= lane ? m1.y : 0.f);
                                }
                            }
                        } else {
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                float m[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int sc = 32 * b + 2 * j + k;
                                    const float q = f32(a[2 * j + k]) * g.d[sc] * ex2((gh - g.hi[sc]) + (glo - g.lo[sc]));
                                    m[k] = 2 * j + k <= lane ? q : 0.f;
                                }
                                o[j] = bf_pair(m[0], m[1]);
                            }
                        }
                    }
                    tmem_st16(tU + 16 * bb, o);   // tU is column 32 hf: M's block 2 hf
                }
                tmem_wait_st();
                tc_fence_before();
                x.arrive(kM + hd);
            }
            if (ok && tiles > 0) ok = finish(tiles - 1);
            // the state that leaves
            void *dst = u.last ? p.hT : nullptr;
            if (ok && dst) {
                const bool fp32 = p.hT_fp32;
                const int64_t e = (static_cast<int64_t>(u.i) * p.H + h) * sn + static_cast<int64_t>(r) * p.P + col;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (fp32)
                        reinterpret_cast<float4 *>(static_cast<float *>(dst) + e)[j] =
                            make_float4(s[2 * j].x, s[2 * j].y, s[2 * j + 1].x, s[2 * j + 1].y);
                    else
                        reinterpret_cast<uint2 *>(static_cast<uint16_t *>(dst) + e)[j] =
                            make_uint2(bf_pair(s[2 * j].x, s[2 * j].y), bf_pair(s[2 * j + 1].x, s[2 * j + 1].y));
                }
            }
        }
    } else if (warp == kIssuer) {
        // ---------------------------------------------------------------- loads of C and B, and the products
        const int bcol = grp * N;
        const uint32_t id_y = idesc_f16(128, 64 * heads, 1, 0, 1);   // C K-major, the states' copies MN-major
        const uint32_t id_u = idesc_f16(128, 64 * heads, 1, 1, 1);   // B^T and the parts of x, both MN-major
        auto load_bc = [&](int i) {
            if (!elect_one()) return;
            const int32_t row = static_cast<int32_t>(start_of(i));
            mbar_arrive_expect_tx(x.bar(kBcFull), 4 * kBlock);
            for (int k = 0; k < 2; ++k) {
                tma_load_2d(base + L::kC + k * kBlock, &maps.c, x.bar(kBcFull), bcol + 64 * k, row);
                tma_load_2d(base + L::kB + k * kBlock, &maps.b, x.bar(kBcFull), bcol + 64 * k, row);
            }
        };
        bool ok = true;
        if (tiles > 0) load_bc(0);
        for (int i = 0; i < tiles && ok; ++i) {
            const uint32_t ph = i & 1, bt = base + L::kB;
            ok = x.met(x.wait(kBcFull, ph));
            if (!ok) break;
            {
                // G: the last tile's has been read (its M is written)
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t o = (k >> 2) * kBlock + (k & 3) * 32;
                        mma_f16(tmem + kColG, smem_desc(base + L::kC + o, 16, 1024, kSwizzle128),
                                smem_desc(bt + o, 16, 1024, kSwizzle128), kIdG, k > 0);
                    }
                    mma_commit(x.bar(kG));
                }
                __syncwarp();
            }
            // both heads side by side, so that C and B^T are read once for the two
            auto product_u = [&](int half) {
                if (elect_one()) {
                    const uint32_t parts = base + L::kParts;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = S - 1; e >= 0; --e)
                            mma_f16(tmem + kColU, smem_desc(bt + (half * 4 + k) * 2048, kBlock, 1024, kSwizzle128),
                                    smem_desc(parts + e * 2 * L::kPart + k * 2048, L::kPart, 1024, kSwizzle128), id_u,
                                    !(half == 0 && k == 0 && e == S - 1));
                    mma_commit(x.bar(half ? kU : kPFree));
                }
                __syncwarp();
            };
            // U takes the place of the last tile's M, which has been multiplied
            for (int hd = 0; hd < heads && ok; ++hd) ok = x.wait(kP0 + hd, ph) && (i == 0 || x.wait(kY + hd, (i - 1) & 1));
            ok = x.met(ok);
            if (!ok) break;
            tc_fence_after();
            product_u(0);
            for (int hd = 0; hd < heads && ok; ++hd) ok = x.wait(kS + hd, ph) && (i == 0 || x.wait(kYFree + hd, (i - 1) & 1));
            ok = x.met(ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_f16(tmem + kColY1, smem_desc(base + L::kC + (k >> 2) * kBlock + (k & 3) * 32, 16, 1024, kSwizzle128),
                            smem_desc(base + L::kState + k * 2048, kBlock, 1024, kSwizzle128), id_y, k > 0);
            }
            __syncwarp();
            for (int hd = 0; hd < heads && ok; ++hd) ok = x.wait(kP1 + hd, ph);
            ok = x.met(ok);
            if (!ok) break;
            tc_fence_after();
            product_u(1);
            if (!ok) break;
            // the last commit covers every product so far: C and B are free
            if (i + 1 < tiles) {
                ok = x.met(x.wait(kU, ph));
                if (!ok) break;
                load_bc(i + 1);
                __syncwarp();
            }
            {
                for (int hd = 0; hd < heads && ok; ++hd) {
                    ok = x.met(x.wait(kM + hd, ph));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t xt = base + L::kX + (hd * 2 + (i & 1)) * kBlock;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_f16_ts(tmem + kColY2 + hd * kColHead, tmem + kColU + hd * kColHead + 8 * k,
                                       smem_desc(xt + k * 2048, kBlock, 1024, kSwizzle128), kIdY, k > 0);
                        mma_commit(x.bar(kY + hd));
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp - kFeeder < heads) {
        // ---------------------------------------------------------------- a head's x and gates, up to two tiles ahead
        const int hd = warp - kFeeder, v = v0 + hd, h = v / slices;
        const Two rate = log2_rate(p.A[h]);
        const float bias = p.dt_bias ? p.dt_bias[h] : 0.f;
        float dt[4];
        bool ok = true;
        if (tiles > 0) load_dt(p, start_of(0), count_of(0), h, dt);
        for (int i = 0; i < tiles; ++i) {
            const int stage = i & 1;
            if (i >= 2) ok = x.met(x.wait(kXFree + hd * 2 + stage, ((i - 2) >> 1) & 1));
            if (!ok) break;
            __syncwarp();
            if (elect_one()) {
                const int bar = kXFull + hd * 2 + stage;
                mbar_arrive_expect_tx(x.bar(bar), kBlock);
                tma_load_2d(base + L::kX + (hd * 2 + stage) * kBlock, &maps.x, x.bar(bar), v * PC,
                            static_cast<int32_t>(start_of(i)));
            }
            __syncwarp();
            const float now[4] = {dt[0], dt[1], dt[2], dt[3]};
            if (i + 1 < tiles) load_dt(p, start_of(i + 1), count_of(i + 1), h, dt);
            make_tc_gates(gates[hd * 2 + stage], now, count_of(i), bias, p.softplus, rate);
#ifdef KDA_TEST_HOOKS
            if (i != g_scan_tc_stall)
#endif
            x.arrive(kGates + hd * 2 + stage);
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
    if (warp == kIssuer) tmem_dealloc(tmem, kCols);
}

template <int S>
cudaError_t launch(const ScanParams &p, int64_t seg, int64_t units, const float *entering, cudaStream_t s) {
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    if (p.rows > 0 && (!encode(&maps.x, p.x, static_cast<int64_t>(p.H) * p.P, p.rows, p.x_stride, TT) ||
                       !encode(&maps.b, p.B, static_cast<int64_t>(p.G) * N, p.rows, p.b_stride, TT) ||
                       !encode(&maps.c, p.C, static_cast<int64_t>(p.G) * N, p.rows, p.c_stride, TT)))
        return cudaErrorInvalidValue;
    cudaError_t err = allow_smem(scan_tc_kernel<S>, Smem<S>::kBytes);
    if (err != cudaSuccess) return err;
    const int64_t pairs = (p.H / p.G * (p.P / PC) + 1) / 2;
    scan_tc_kernel<S><<<static_cast<unsigned>(units * p.G * pairs), NT, Smem<S>::kBytes, s>>>(p, maps, seg, entering);
    return cudaGetLastError();
}

}  // namespace tc
}  // namespace scan

cudaError_t launch_scan_tc(const ScanParams &p, int64_t seg, int64_t units, const float *entering, cudaStream_t s) {
    using namespace scan::tc;
    return p.hT && p.hT_fp32 ? launch<3>(p, seg, units, entering, s) : launch<2>(p, seg, units, entering, s);
}

cudaError_t read_and_clear_scan_tc_error(unsigned int *value) {
    cudaError_t err = cudaMemcpyFromSymbol(value, scan::tc::g_scan_tc_error, sizeof(*value));
    if (err != cudaSuccess || *value == 0) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(scan::tc::g_scan_tc_error, &zero, sizeof(zero));
}

#ifdef KDA_TEST_HOOKS
extern "C" int kda_test_set_scan_tc_stall(int at) {
    return static_cast<int>(cudaMemcpyToSymbol(scan::tc::g_scan_tc_stall, &at, sizeof(int)));
}
#endif

}  // namespace kda
