// kda_scan_tc_state.cu -- the scan's state alone on tcgen05, sm_100a.
//
// Two uses: what each piece of a cut sequence adds to the state (kda_scan_fwd.cu), and, for the backward, the
// state S entering every tile of 128 tokens and the gradient R of the state leaving it:
//
//   S_end = e^(Gamma_end) S_0 + B^T Diag(d e^(Gamma_end - Gamma)) x          tiles in order
//   R_0   = e^(Gamma_end) R_end + C^T Diag(e^Gamma) dy                       tiles backwards (blockIdx.y 1)
//
// per 64 columns of a head, U = rows^T Diag(weight) cols being one tcgen05 product (128 x 64, K 128; at a state size of 64
// half of its rows are of no use, but the product is not what bounds it), with the
// weighted columns in S bf16 parts (three: 24 bits). The state stays fp32 in the registers of 256 threads.
//
// A CTA takes two heads of a group side by side: one product with N = 128 reads the rows once for both, 64 cycles per
// K step and part instead of 2 x 48, 1536 per tile with three parts. Eight warps per head form the parts of the next tile,
// half by half, while this one's product runs, then add U to the state; four warps run ahead with gates and loads. Bound
// by the elements' chain: parts, fence, U, state. (65536 tokens x 32 heads x 128, two parts: 227 us, 4000 cycles for two
// heads' tile; with tiles of 64 tokens 277. 2 x 4096 tokens x 64 heads x 64, both directions, every tile's states stored:
// 114 us; 123. The same of 5 packed sequences, 3802 tokens x 32 heads x 128, state size 64: 69 us; warp-level products, 77.)
//
// Every wait is bounded; one that runs out raises kErrTimeout and winds the CTA down.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_scan_tc.cuh"

namespace kda {
namespace scan {
namespace tc {

__device__ unsigned int g_scan_state_error = 0;
#ifdef KDA_TEST_HOOKS
// Test-only build (never the product library): the gates of this tile of every CTA are not signalled, so that the bounded
// waits for them run out.
__device__ int g_scan_tc_state_stall = -1;
#endif

constexpr int kIssuer = 16, kFeeder = 17, NT = 32 * 21;
constexpr int TT = kScanTcTile;

struct StateGates {
    float weight[TT];
    float total;
    float pad[3];
};

struct StateRest {
    Two decay[4];
    uint32_t tmem, abort;
};

constexpr uint32_t kHalf = 64 * 128;      // 64 rows of 128 bytes
template <int S>
struct StateSmem {
    static constexpr uint32_t kRows = 0;                                   // [stage] 128 x 128: two blocks of columns
    static constexpr uint32_t kCols = kRows + 4 * kBlock;                  // [head][stage]
    static constexpr uint32_t kParts = kCols + 4 * kBlock;                 // [half][S][head] 64 tokens
    static constexpr uint32_t kGates = kParts + 2 * S * 2 * kHalf;         // [head][stage]
    static constexpr uint32_t kBars = kGates + 4 * sizeof(StateGates);
    static constexpr uint32_t kRest = kBars + 8 * 20;                      // StateRest
    static constexpr uint32_t kBytes = kRest + 64;
    static_assert(kBytes <= 227 * 1024, "shared memory of one CTA");
};

enum : int {
    kRowsFull = 0,      // [stage]
    kColsFull = 2,      // [head][stage]
    kGatesFull = 6,     // [head][stage]
    kPFree = 10,        // the first half's product is done
    kU = 11,            // [stage] the tile's products are done
    kColsFree = 13,     // [head][stage], the head's eight warps: the columns and gates have been used
    kParts = 17,        // [half], all element warps: the parts are written
    kBarCount = 19
};

struct StateMaps {
    CUtensorMap rows[2], cols[2];   // B and x; C and dy
};

// NS: state size. At 64 the products' upper 64 rows are of no use (their operand is whatever lies there).
template <int S, int NS>
__global__ void __launch_bounds__(NT, 1)
    scan_state_tc_kernel(ScanParams p, const __grid_constant__ StateMaps maps, int64_t seg, ScanStateRun run0,
                         ScanStateRun run1) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = StateSmem<S>;
    const uint32_t base = smem_u32(smem);
    StateRest &rest = *reinterpret_cast<StateRest *>(smem + L::kRest);
    Ctx x;
    x.bars = base + L::kBars;
    x.abort = &rest.abort;
    x.error = &g_scan_state_error;
    StateGates *gates = reinterpret_cast<StateGates *>(smem + L::kGates);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seqs, &g_scan_state_error);

    const bool rev = blockIdx.y == 1;
    const ScanStateRun &run = rev ? run1 : run0;
    const int slices = p.P / PC, per_group = p.H / p.G * slices, pairs = (per_group + 1) / 2;
    const int64_t unit = blockIdx.x / (p.G * pairs);
    const int gp = static_cast<int>(blockIdx.x % (p.G * pairs)), grp = gp / pairs, in_group = gp % pairs * 2;
    const int v0 = grp * per_group + in_group, heads = in_group + 1 < per_group ? 2 : 1;
    const Piece u = find_piece(p.seqs, unit, seg);
    const bool head = rev ? u.last : u.first, tail = rev ? u.first : u.last;
    if (u.none || (run.leave && tail)) return;
    const int64_t lo = u.a / TT;
    const int tiles = static_cast<int>(u.b > u.a ? (u.b + TT - 1) / TT - lo : 0);
    auto cell = [&](int i) { return rev ? lo + tiles - 1 - i : lo + i; };
    auto start_of = [&](int i) { return cell(i) * TT > u.a ? cell(i) * TT : u.a; };
    auto count_of = [&](int i) {
        const int64_t e = (cell(i) + 1) * TT < u.b ? (cell(i) + 1) * TT : u.b;
        return static_cast<int>(e - start_of(i));
    };

    if (warp == kIssuer) {
        if (lane == 0) {
            for (int i = 0; i < kBarCount; ++i) mbar_init(x.bar(i), i < kColsFree ? 1 : i < kParts ? 8 : 8 * heads);
            rest.abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(smem_u32(&rest.tmem), 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = rest.tmem;

    if (warp < kIssuer) {
        // ---------------------------------------------------------------- a head's elements
        // warp: rows 32 wq .. + 32 of the state, columns 32 hf .. + 32, in the layout of tmem_ld_frag: a quad of threads
        // then has 32 bytes of a row, and the state goes to memory as it is
        const int hd = warp >> 3, hf = (warp >> 2) & 1, wq = warp & 3, t256 = tid & 255;
        if (hd < heads) {
            const int v = v0 + hd, h = v / slices, col = v % slices * PC + 32 * hf;
            const uint32_t tU = tmem + hd * 64 + 32 * hf + (static_cast<uint32_t>(wq * 32) << 16);
            const bool mine = wq * 32 < NS;
            const int64_t sn = static_cast<int64_t>(NS) * p.P, at_r = static_cast<int64_t>(wq * 32 + (lane >> 2)) * p.P + col + (lane & 3) * 2;
            float2 s[16];   // [8 i + 2 j + k]: row 16 i + 8 k + lane / 4, columns 8 j + 2 (lane % 4) and the next
            auto place = [&](int m) { return static_cast<int64_t>((m >> 3) * 16 + (m & 1) * 8) * p.P + ((m >> 1) & 3) * 8; };
            {
                const void *init = rev ? static_cast<const void *>(p.dhT) : p.h0;
                const void *src = !mine ? nullptr : run.entering ? run.entering : head && !run.leave ? init : nullptr;
                const bool fp32 = run.entering || rev || p.h0_fp32;
                const int64_t e = ((run.entering ? unit : static_cast<int64_t>(u.i)) * p.H + h) * sn + at_r;
#pragma unroll
                for (int m = 0; m < 16; ++m) {
                    s[m] = make_float2(0.f, 0.f);
                    if (src && fp32) {
                        s[m] = *reinterpret_cast<const float2 *>(static_cast<const float *>(src) + e + place(m));
                    } else if (src) {
                        const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(src) + e + place(m));
                        s[m] = make_float2(bf_low(w), bf_high(w));
                    }
                }
            }
            auto store = [&](float *dst) {
#pragma unroll
                for (int m = 0; m < 16; ++m) *reinterpret_cast<float2 *>(dst + place(m)) = s[m];
            };
            float total = 0.f, next_total = 0.f;
            // the weighted columns of half a tile in parts; four threads per token
            auto write_parts = [&](int i, int half) {
                const int cnt = count_of(i), st = i & 1, row = half * 64 + (t256 >> 2);
                const uint32_t ph = (i >> 1) & 1;
                if (half == 0) {
                    if (!x.met(x.wait(kColsFull + hd * 2 + st, ph) && x.wait(kGatesFull + hd * 2 + st, ph))) return false;
                    if (cnt < TT && hd == 0) {
                        // rows behind the piece: whatever they hold would multiply zeros below
                        if (!x.met(x.wait(kRowsFull + st, ph))) return false;
                        uint8_t *rt = smem + L::kRows + st * 2 * kBlock + (t256 & 1) * kBlock + (t256 >> 1) * 128;
                        if ((t256 >> 1) >= cnt && (t256 & 1) < NS / 64)
#pragma unroll
                            for (int j = 0; j < 8; ++j) sts(rt + j * 16, make_uint4(0u, 0u, 0u, 0u));
                    }
                }
                // the last tile's have been multiplied
                if (i > 0 && !x.met(half ? x.wait(kU + (st ^ 1), ((i - 1) >> 1) & 1) : x.wait(kPFree, (i - 1) & 1))) return false;
                const StateGates &g = gates[hd * 2 + st];
                const uint8_t *ct = smem + L::kCols + (hd * 2 + st) * kBlock;
                uint8_t *parts = smem + L::kParts + half * S * 2 * kHalf + hd * kHalf;
                const float w = g.weight[row];
                next_total = g.total;
                const float2 w2 = make_float2(w, w), minus1 = make_float2(-1.f, -1.f);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int chunk = (t256 & 3) * 2 + j;   // two rows' chunks of a turn lie in different banks
                    uint32_t o[S][4];
                    if (row < cnt) {
                        const uint4 q = lds(ct + sw128(row, chunk));
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
#pragma unroll
                        for (int e = 0; e < S; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0u;
                    }
#pragma unroll
                    for (int e = 0; e < S; ++e)
                        sts(parts + e * 2 * kHalf + sw128(t256 >> 2, chunk), make_uint4(o[e][0], o[e][1], o[e][2], o[e][3]));
                }
                fence_proxy_async_smem();
                tc_fence_before();
                x.arrive(kParts + half);
                if (half) x.arrive(kColsFree + hd * 2 + st);
                return true;
            };
            bool ok = tiles == 0 || (write_parts(0, 0) && write_parts(0, 1));
            for (int i = 0; i < tiles && ok; ++i) {
                total = next_total;
                if (i + 1 < tiles) ok = write_parts(i + 1, 0) && write_parts(i + 1, 1);
                if (!ok) break;
                if (run.states && mine) store(run.states + ((u.i + cell(i)) * p.H + h) * sn + at_r);
                ok = x.met(x.wait(kU + (i & 1), (i >> 1) & 1));
                if (!ok) break;
                if (!mine) continue;
                tc_fence_after();
                uint32_t a[2][16];
                tmem_ld_frag(tU + (i & 1) * 128, a[0]);
                tmem_ld_frag(tU + (i & 1) * 128 + (16u << 16), a[1]);
                const float2 tot = make_float2(total, total);
                tmem_wait_ld();
#pragma unroll
                for (int m = 0; m < 16; ++m)
                    s[m] = fma2(s[m], tot, make_float2(f32(a[m >> 3][2 * (m & 7)]), f32(a[m >> 3][2 * (m & 7) + 1])));
            }
            float *dst = !mine ? nullptr : run.leave ? run.leave : rev && tail ? p.dh0 : nullptr;
            if (ok && dst) store(dst + ((run.leave ? unit : static_cast<int64_t>(u.i)) * p.H + h) * sn + at_r);
        }
    } else if (warp == kIssuer) {
        // ---------------------------------------------------------------- loads of the rows, and the products
        auto load_rows = [&](int i) {
            if (elect_one()) {
                const int st = i & 1;
                const uint32_t bar = x.bar(kRowsFull + st), dst = base + L::kRows + st * 2 * kBlock;
                const int32_t row = static_cast<int32_t>(start_of(i));
                mbar_arrive_expect_tx(bar, NS / 64 * kBlock);
                for (int k = 0; k < NS / 64; ++k) tma_load_2d(dst + k * kBlock, &maps.rows[rev], bar, grp * NS + 64 * k, row);
            }
            __syncwarp();
        };
        const uint32_t id = idesc_f16(128, heads == 2 ? 128 : 64, 1, 1, 1);
        bool ok = true;
        for (int i = 0; i < 2 && i < tiles; ++i) load_rows(i);
        for (int i = 0; i < tiles && ok; ++i) {
            const int st = i & 1;
            const bool rows = x.wait(kRowsFull + st, (i >> 1) & 1);
            for (int half = 0; half < 2 && ok; ++half) {
                ok = x.met(rows && x.wait(kParts + half, i & 1));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t rt = base + L::kRows + st * 2 * kBlock + half * 4 * 2048;
                    const uint32_t parts = base + L::kParts + half * S * 2 * kHalf;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = S - 1; e >= 0; --e)
                            mma_f16(tmem + st * 128, smem_desc(rt + k * 2048, kBlock, 1024, kSwizzle128),
                                    smem_desc(parts + e * 2 * kHalf + k * 2048, kHalf, 1024, kSwizzle128), id,
                                    !(half == 0 && k == 0 && e == S - 1));
                    mma_commit(x.bar(half ? kU + st : kPFree));
                }
                __syncwarp();
            }
            if (ok && i + 2 < tiles) {
                ok = x.met(x.wait(kU + st, (i >> 1) & 1));   // this tile's rows have been multiplied
                if (!ok) break;
                load_rows(i + 2);
            }
        }
    } else {
        // ---------------------------------------------------------------- a head's gates and columns, every other tile
        const int f = warp - kFeeder, hd = f >> 1, v = v0 + hd, t4 = 4 * lane;
        if (hd < heads) {
            const int h = v / slices;
            const Two rate = log2_rate(p.A[h]);
            const float bias = p.dt_bias ? p.dt_bias[h] : 0.f;
            Two decay = {0.f, 0.f};
            bool ok = true;
            float dt[4] = {0.f, 0.f, 0.f, 0.f};
            auto steps = [&](int i) {
                const int cnt = count_of(i);
                const float *src = p.dt + start_of(i) * p.H + h;
#pragma unroll
                for (int j = 0; j < 4; ++j) dt[j] = t4 + j < cnt ? src[static_cast<int64_t>(t4 + j) * p.H] : 0.f;
            };
            if ((f & 1) < tiles) steps(f & 1);
            for (int i = f & 1; i < tiles; i += 2) {
                const int st = i & 1, cnt = count_of(i);
                if (i >= 2) ok = x.met(x.wait(kColsFree + hd * 2 + st, ((i - 2) >> 1) & 1));
                if (!ok) break;
                __syncwarp();
                if (elect_one()) {
                    const int bar = kColsFull + hd * 2 + st;
                    mbar_arrive_expect_tx(x.bar(bar), kBlock);
                    tma_load_2d(base + L::kCols + (hd * 2 + st) * kBlock, &maps.cols[rev], x.bar(bar), v * PC,
                                static_cast<int32_t>(start_of(i)));
                }
                __syncwarp();
                StateGates &g = gates[hd * 2 + st];
                float d[4], w[4];
                Two c[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float arg;
                    d[j] = t4 + j < cnt ? step_of(dt[j], bias, p.softplus, &arg) : 0.f;
                    c[j] = t4 + j < cnt ? log_decay(d[j], rate) : Two{0.f, 0.f};
                    if (j) c[j] = c[j - 1] + c[j];
                }
                if (i + 2 < tiles) steps(i + 2);
                const Two sum = scan_lanes(c[3]), all = shfl(sum, 31);
                Two before = {__shfl_up_sync(0xffffffffu, sum.hi, 1), __shfl_up_sync(0xffffffffu, sum.lo, 1)};
                if (lane == 0) before = {0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Two at = before + c[j];
                    w[j] = rev ? ex2(at) : d[j] * ex2(minus(all, at));
                }
                reinterpret_cast<float4 *>(g.weight)[lane] = make_float4(w[0], w[1], w[2], w[3]);
                if (lane == 0) g.total = ex2(all);
                decay = decay + all;
#ifdef KDA_TEST_HOOKS
                if (i != g_scan_tc_state_stall)
#endif
                x.arrive(kGatesFull + hd * 2 + st);
            }
            if (lane == 0) rest.decay[f] = decay;
        }
    }
    if (rest.abort) {
        // copies may still be in flight into this CTA's shared memory
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 20000000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc(tmem, 256);
    if (run.leave && tid < heads && (v0 + tid) % slices == 0)
        run.leave_decay[unit * p.H + (v0 + tid) / slices] = ex2(rest.decay[2 * tid] + rest.decay[2 * tid + 1]);
}

template <int S, int NS>
cudaError_t state_launch(const ScanParams &p, int directions, int64_t seg, int64_t units, const ScanStateRun &fwd,
                         const ScanStateRun &rev, cudaStream_t s) {
    StateMaps maps;
    memset(&maps, 0, sizeof(maps));
    const int64_t hp = static_cast<int64_t>(p.H) * p.P, gn = static_cast<int64_t>(p.G) * NS;
    if (p.rows > 0 && (!encode(&maps.rows[0], p.B, gn, p.rows, p.b_stride, TT) ||
                       !encode(&maps.cols[0], p.x, hp, p.rows, p.x_stride, TT) ||
                       (directions > 1 && (!encode(&maps.rows[1], p.C, gn, p.rows, p.c_stride, TT) ||
                                           !encode(&maps.cols[1], p.dout, hp, p.rows, p.dout_stride, TT)))))
        return cudaErrorInvalidValue;
    cudaError_t err = allow_smem(scan_state_tc_kernel<S, NS>, StateSmem<S>::kBytes);
    if (err != cudaSuccess) return err;
    const int64_t pairs = (p.H / p.G * (p.P / PC) + 1) / 2;
    const dim3 grid(static_cast<unsigned>(units * p.G * pairs), static_cast<unsigned>(directions));
    scan_state_tc_kernel<S, NS><<<grid, NT, StateSmem<S>::kBytes, s>>>(p, maps, seg, fwd, rev);
    return cudaGetLastError();
}

}  // namespace tc
}  // namespace scan

cudaError_t launch_scan_tc_state(const ScanParams &p, int parts, int directions, int64_t seg, int64_t units,
                                 const ScanStateRun &fwd, const ScanStateRun &rev, cudaStream_t s) {
    using namespace scan::tc;
    return scan::by_state(p.N, [&](auto n) {
        constexpr int NS = decltype(n)::value;
        return parts == 3 ? state_launch<3, NS>(p, directions, seg, units, fwd, rev, s)
                          : state_launch<2, NS>(p, directions, seg, units, fwd, rev, s);
    });
}

cudaError_t read_and_clear_scan_state_error(unsigned int *value) {
    cudaError_t err = cudaMemcpyFromSymbol(value, scan::tc::g_scan_state_error, sizeof(*value));
    if (err != cudaSuccess || *value == 0) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(scan::tc::g_scan_state_error, &zero, sizeof(zero));
}

#ifdef KDA_TEST_HOOKS
extern "C" int kda_test_set_scan_tc_state_stall(int at) {
    return static_cast<int>(cudaMemcpyToSymbol(scan::tc::g_scan_tc_state_stall, &at, sizeof(int)));
}
#endif

}  // namespace kda
