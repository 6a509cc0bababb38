// kda_seq.cuh -- packed sequences on the device, and small conversions, shared by the convolution,
// q/k and scan kernels.
//
// A call's rows are the tokens of `n` sequences one behind the other: batch rows of `len` tokens
// each (cu == nullptr) or packed ones behind the offsets cu[0 .. n]. Offsets are clamped into
// [0, len] and the first sequence begins at 0 whatever cu[0] holds, so that every row has a sequence that
// begins at or before it: a malformed table makes wrong results but no access out of bounds. check_offsets
// raises the error bit for it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"

namespace kda {

struct Seqs {
    const int32_t *cu;   // device, n + 1 offsets, or nullptr
    int32_t n;
    int64_t len;         // tokens per batch row, or of the packed total

    __device__ __forceinline__ int64_t begin(int32_t i) const {
        if (!cu) return static_cast<int64_t>(i) * len;
        const int64_t c = i ? cu[i] : 0;
        return c < 0 ? 0 : (c > len ? len : c);
    }
    // never before begin(i)
    __device__ __forceinline__ int64_t end(int32_t i) const {
        if (!cu) return static_cast<int64_t>(i + 1) * len;
        const int64_t b = begin(i), e = begin(i + 1);
        return e < b ? b : e;
    }
};

// The largest i in [0, n) with key(i) <= u, by all 32 lanes of a converged warp (key(0) <= u is
// taken for granted): each step probes 32 places at once, so 1024 sequences take two dependent
// loads. `key` is non-decreasing for a well-formed table; for any other the answer is some i in range.
template <class Key>
__device__ __forceinline__ int32_t warp_upper(int32_t n, int64_t u, Key key) {
    int32_t lo = 0, hi = n;
    const int lane = threadIdx.x & 31;
    while (hi - lo > 1) {
        const int32_t step = (hi - lo + 31) >> 5;
        const int32_t m = lo + lane * step;
        const bool ok = lane == 0 || (m < hi && key(m) <= u);
        const unsigned b = __ballot_sync(0xffffffffu, ok);
        lo += (31 - __clz(b)) * step;
        if (lo + step < hi) hi = lo + step;
    }
    return lo;
}

// Raise kErrCuSeqlens in *word unless the offsets run 0, ..., <= len without decreasing. Called by
// one whole CTA of a launch.
__device__ __forceinline__ void check_offsets(const Seqs &s, unsigned int *word) {
    if (!s.cu) return;
    bool bad = false;
    for (int32_t i = threadIdx.x; i <= s.n; i += blockDim.x) {
        const int32_t c = s.cu[i], before = i ? s.cu[i - 1] : 0;
        bad |= c < before || c > s.len || (i == 0 && c != 0);
    }
    if (bad) atomicOr(word, kErrCuSeqlens);
}

__device__ __forceinline__ float bf_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf_pair(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

// pairs of fp32 in one instruction (sm_100's f32x2)
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// V consecutive elements as floats; T is float or __nv_bfloat16; loads and stores of 16 bytes (8 for four bf16).
template <class T, int V>
struct Vec;
template <int V>
struct Vec<__nv_bfloat16, V> {
    uint4 raw[V / 8];
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + at);
#pragma unroll
        for (int i = 0; i < V / 8; ++i) raw[i] = s[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < V / 8; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < V / 8; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[8 * i + 2 * j] = bf_low(w[j]);
                x[8 * i + 2 * j + 1] = bf_high(w[j]);
            }
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, const float (&x)[V]) {
        uint4 *d = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + at);
#pragma unroll
        for (int i = 0; i < V / 8; ++i)
            d[i] = make_uint4(bf_pair(x[8 * i], x[8 * i + 1]), bf_pair(x[8 * i + 2], x[8 * i + 3]),
                              bf_pair(x[8 * i + 4], x[8 * i + 5]), bf_pair(x[8 * i + 6], x[8 * i + 7]));
    }
};
template <>
struct Vec<__nv_bfloat16, 4> {
    uint2 raw;
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        raw = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + at);
    }
    __device__ __forceinline__ void zero() { raw = make_uint2(0u, 0u); }
    __device__ __forceinline__ void get(float (&x)[4]) const {
        x[0] = bf_low(raw.x);
        x[1] = bf_high(raw.x);
        x[2] = bf_low(raw.y);
        x[3] = bf_high(raw.y);
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, const float (&x)[4]) {
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p) + at) =
            make_uint2(bf_pair(x[0], x[1]), bf_pair(x[2], x[3]));
    }
};
template <int V>
struct Vec<float, V> {
    float4 raw[V / 4];
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) raw[i] = s[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) raw[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            x[4 * i] = raw[i].x;
            x[4 * i + 1] = raw[i].y;
            x[4 * i + 2] = raw[i].z;
            x[4 * i + 3] = raw[i].w;
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, const float (&x)[V]) {
        float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) d[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
};

}  // namespace kda
