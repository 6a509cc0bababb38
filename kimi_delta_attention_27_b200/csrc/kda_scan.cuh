// kda_scan.cuh -- what the scan's kernels share: gates of a tile, tiles in shared memory, warp-level matrix products.
#pragma once

#include "kda_scan.h"

namespace kda {
namespace scan {

constexpr int T = kScanTile;      // tokens per tile
constexpr int PC = 64;            // head channels per CTA (the columns of the state do not mix)
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2eHi = 1.44269502f, kLog2eLo = static_cast<float>(1.4426950408889634 - 1.44269502162933349609375);
constexpr float kMinLog2 = -1442.695f;   // log2(e^-1000)

__device__ __forceinline__ float ex2(float y) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return r;
}

// the step d = dt or softplus(dt + bias); u returns the argument
__device__ __forceinline__ float step_of(float dt, float bias, int softplus, float *u) {
    *u = dt + bias;
    return softplus ? fmaxf(*u, 0.f) + log1pf(expf(-fabsf(*u))) : *u;
}

// Sums of log decays are kept as two floats hi + lo (about 48 bits), added by error-free sums: the difference
// of two of them, which is what the kernels exponentiate, then has the relative error of one 32-bit
// rounding however large the sums are. (In fp64, which this GPU has little of, the same sums took most of a tile's time.)
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two operator+(Two a, Two b) {
    const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
    const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
    const float l = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
    const float hi = __fadd_rn(s, l);
    return {hi, __fsub_rn(l, __fsub_rn(hi, s))};
}
__device__ __forceinline__ float minus(Two a, Two b) { return (a.hi - b.hi) + (a.lo - b.lo); }
__device__ __forceinline__ Two shfl(Two v, int from) {
    return {__shfl_sync(0xffffffffu, v.hi, from), __shfl_sync(0xffffffffu, v.lo, from)};
}
// the sums over lanes 0 .. l
__device__ __forceinline__ Two scan_lanes(Two v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const Two o = {__shfl_up_sync(0xffffffffu, v.hi, k), __shfl_up_sync(0xffffffffu, v.lo, k)};
        const Two w = o + v;
        if (lane >= k) v = w;
    }
    return v;
}
// log2 of a step's decay, d A log2(e). A step whose decay is below e^-1000 leaves nothing of the state even in
// 64 bits; the floor keeps the sums exact enough where one step of a tile decays by 10^30. Only numbers below it are
// replaced: a NaN, of A or of the step, stays one.
__device__ __forceinline__ Two log_decay(float d, Two a2) {
    const float hi = d * a2.hi, lo = fmaf(d, a2.hi, -hi) + d * a2.lo;
    return hi <= kMinLog2 ? Two{kMinLog2, 0.f} : Two{hi, lo};
}
// A log2(e) to two floats
__device__ __forceinline__ Two log2_rate(float A) {
    const float hi = A * kLog2eHi;
    return {hi, fmaf(A, kLog2eHi, -hi) + A * kLog2eLo};
}
// 2^v
__device__ __forceinline__ float ex2(Two v) { return ex2(v.hi) * fmaf(v.lo, kLn2, 1.f); }

// A tile's gates, in powers of two.
struct Gates {
    float hi[T], lo[T];   // log2 of the decay from the tile's start through token t
    float d[T];           // the steps
    float from[T];        // decay from the tile's start through t
    float weight[T];      // d times the decay from t (exclusive) to the tile's end
    float total;          // decay of the whole tile
    float pad[3];
};

// By one warp: lane l has tokens 2l and 2l + 1 of cnt (steps d0, d1; 0 behind the tile's last token, where nothing
// decays whatever A is).
__device__ __forceinline__ void make_gates(Gates &g, float d0, float d1, int cnt, float A) {
    const int lane = threadIdx.x & 31;
    const Two a2 = log2_rate(A), none = {0.f, 0.f};
    const Two l0 = 2 * lane < cnt ? log_decay(d0, a2) : none, l1 = 2 * lane + 1 < cnt ? log_decay(d1, a2) : none;
    const Two s = scan_lanes(l0 + l1), total = shfl(s, 31);
    // through the lane's first token: the sum through the lane before, and its own
    const Two before = {__shfl_up_sync(0xffffffffu, s.hi, 1), __shfl_up_sync(0xffffffffu, s.lo, 1)};
    const Two c[2] = {lane ? before + l0 : l0, s};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = 2 * lane + j;
        const float d = j ? d1 : d0;
        g.hi[t] = c[j].hi;
        g.lo[t] = c[j].lo;
        g.d[t] = d;
        g.from[t] = ex2(c[j]);
        g.weight[t] = d * ex2(minus(total, c[j]));
    }
    if (lane == 0) g.total = ex2(total);
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// byte offset of (row, 16-byte chunk) in a tile of ROWB-byte rows: the chunk's low three bits are
// exchanged with the row's, so that the eight rows of an 8 x 8 matrix lie in different banks
template <int ROWB>
__device__ __forceinline__ uint32_t at(int row, int chunk) {
    return static_cast<uint32_t>(row * ROWB + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    const int bytes = valid ? 16 : 0;   // 0: the 16 bytes are filled with zeros and nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// `cnt` rows (of T) of ROWB bytes from src (stride in elements) into a swizzled tile; the rest zero
template <int ROWB, int NT>
__device__ __forceinline__ void load_tile(uint32_t dst, const uint16_t *src, int64_t stride, int cnt) {
    constexpr int CH = ROWB / 16;
#pragma unroll
    for (int j = 0; j < T * CH / NT; ++j) {
        const int e = j * NT + threadIdx.x, r = e / CH, c = e % CH;
        const bool ok = r < cnt;
        cp_async16(dst + at<ROWB>(r, c), src + (ok ? r : 0) * stride + c * 8, ok);
    }
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// 16 x 16 fragments. A: rows [r0, +16), columns 8 * c0 .. + 16 of a row-major tile.
template <int ROWB>
__device__ __forceinline__ void frag_a(uint32_t tile, int r0, int c0, uint32_t (&f)[4]) {
    const int l = threadIdx.x & 31;
    ldsm4(tile + at<ROWB>(r0 + (l & 15), c0 + (l >> 4)), f);
}
// A of the transposed tile: A's rows are the tile's columns 8 * c0 .. + 16, its columns the tile's rows [r0, +16)
template <int ROWB>
__device__ __forceinline__ void frag_at(uint32_t tile, int r0, int c0, uint32_t (&f)[4]) {
    const int l = threadIdx.x & 31;
    ldsm4t(tile + at<ROWB>(r0 + (l & 7) + ((l >> 4) << 3), c0 + ((l >> 3) & 1)), f);
}
// B (k x n) of two 8-column tiles, n from the tile's rows [r0, +16), k its columns 8 * c0 .. + 16:
// f[0], f[1] the first n-tile, f[2], f[3] the second
template <int ROWB>
__device__ __forceinline__ void frag_b(uint32_t tile, int r0, int c0, uint32_t (&f)[4]) {
    const int l = threadIdx.x & 31;
    ldsm4(tile + at<ROWB>(r0 + (l & 7) + ((l >> 4) << 3), c0 + ((l >> 3) & 1)), f);
}
// B with k from the tile's rows [r0, +16) and n its columns 8 * c0 .. + 16
template <int ROWB>
__device__ __forceinline__ void frag_bt(uint32_t tile, int r0, int c0, uint32_t (&f)[4]) {
    const int l = threadIdx.x & 31;
    ldsm4t(tile + at<ROWB>(r0 + (l & 15), c0 + (l >> 4)), f);
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// v = hi + mid + lo to 24 bits, each part exact in bf16 (the rounding of a part goes into the next)
template <int S>
__device__ __forceinline__ void split(float v0, float v1, uint32_t (&part)[S]) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
        part[s] = bf_pair(v0, v1);
        v0 -= bf_low(part[s]);
        v1 -= bf_high(part[s]);
    }
}

constexpr int64_t kWhole = 0xffffffffLL;   // one cell: pieces are whole sequences

struct Piece {
    int32_t i;            // sequence
    int64_t a, b;         // its tokens [a, b)
    bool first, last, none;
};

// the cell of `seg` tokens that token x lies in; both below 2^32, where a division is a third as long
__device__ __forceinline__ int64_t cell_of(int64_t x, int64_t seg) {
    return static_cast<uint32_t>(x) / static_cast<uint32_t>(seg);
}

// The sequence with `rank` longer ones before it (of n <= 64; equal lengths in order), by a converged warp: whole
// sequences are worked on longest first.
__device__ __forceinline__ int32_t by_length(const Seqs &s, int32_t rank) {
    const int lane = threadIdx.x & 31;
    int64_t mine[2];
    int before[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) mine[k] = lane + 32 * k < s.n ? s.end(lane + 32 * k) - s.begin(lane + 32 * k) : -1;
    for (int j = 0; j < s.n; ++j) {
        const int64_t other = __shfl_sync(0xffffffffu, j < 32 ? mine[0] : mine[1], j & 31);
#pragma unroll
        for (int k = 0; k < 2; ++k) before[k] += other > mine[k] || (other == mine[k] && j < lane + 32 * k);
    }
    const unsigned lo = __ballot_sync(0xffffffffu, before[0] == rank && lane < s.n);
    const unsigned hi = __ballot_sync(0xffffffffu, before[1] == rank && lane + 32 < s.n);
    return lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
}

// piece `u` on the grid of `seg` tokens; a sequence's first and last pieces may be empty
__device__ __forceinline__ Piece find_piece(const Seqs &s, int64_t u, int64_t seg) {
    Piece p;
    if (seg == kWhole && s.cu && s.n <= 64) {
        p.i = by_length(s, static_cast<int32_t>(u));
        p.first = p.last = true;
        p.none = false;
        p.a = s.begin(p.i);
        p.b = s.end(p.i);
        return p;
    }
    p.i = warp_upper(s.n, u, [&](int32_t j) { return j + cell_of(s.begin(j), seg); });
    const int64_t c = u - p.i, sb = s.begin(p.i), se = s.end(p.i), cb = cell_of(sb, seg), ce = cell_of(se, seg);
    p.none = c < cb || c > ce;
    p.first = c == cb;
    p.last = c == ce;
    p.a = p.first ? sb : c * seg;
    p.b = p.last ? se : (c + 1) * seg;
    return p;
}

// the steps of a lane's two tokens of the tile [start, start + cnt)
__device__ __forceinline__ void load_steps(const ScanParams &p, int64_t start, int cnt, int h, float &d0, float &d1) {
    const int t = 2 * (threadIdx.x & 31);
    const float bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    float u;
    d0 = t < cnt ? step_of(p.dt[(start + t) * p.H + h], bias, p.softplus, &u) : 0.f;
    d1 = t + 1 < cnt ? step_of(p.dt[(start + t + 1) * p.H + h], bias, p.softplus, &u) : 0.f;
}

// cell c of 64 tokens, cut to the piece
__device__ __forceinline__ int64_t tile_start(const Piece &u, int64_t c) { return c * T > u.a ? c * T : u.a; }
__device__ __forceinline__ int tile_count(const Piece &u, int64_t c) {
    const int64_t e = (c + 1) * T < u.b ? (c + 1) * T : u.b;
    return static_cast<int>(e - tile_start(u, c));
}

template <class F>
cudaError_t by_state(int N, F f) {
    return N == 64 ? f(std::integral_constant<int, 64>()) : f(std::integral_constant<int, 128>());
}

template <class K>
cudaError_t allow_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace scan
}  // namespace kda
