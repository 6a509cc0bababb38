// kda_scan_tc.cuh -- what the scan's tcgen05 kernels share: PTX wrappers, bounded waits, tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <string.h>

#include "kda_scan.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace scan {
namespace tc {

using namespace ptx;

constexpr int N = 128;                    // state size
constexpr uint32_t kBlock = 16384;        // 128 rows of 128 bytes: 64 bf16 columns
#ifdef KDA_TEST_HOOKS
constexpr uint64_t kWaitLimitNs = 100000000ull;    // 100 ms in the test-only build
#else
constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s: far above any legitimate wait
#endif

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// 16 lanes x 32 columns in the layout of a warp-level product's accumulators: r[4 j + 2 i + e] is row lane / 4 + 8 i,
// column 8 j + 2 (lane % 4) + e
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ uint4 lds(const uint8_t *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void sts(uint8_t *p, uint4 v) { *reinterpret_cast<uint4 *>(p) = v; }
__device__ __forceinline__ float f32(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t sw128(int r, int j) { return static_cast<uint32_t>(r * 128 + ((j ^ (r & 7)) << 4)); }
// bit b: any of the eight lanes of block b of 32 tokens, of a ballot
__device__ __forceinline__ uint32_t steep_blocks(unsigned ballot) {
    return (ballot & 0xffu ? 1u : 0u) | (ballot & 0xff00u ? 2u : 0u) | (ballot & 0xff0000u ? 4u : 0u) |
           (ballot & 0xff000000u ? 8u : 0u);
}
// Whether the phase of the given parity has completed. Acquire at CTA scope: nothing here comes from another CTA.
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

struct Ctx {
    uint32_t bars;
    volatile uint32_t *abort;   // in shared memory
    unsigned int *error;        // the device error word of the kernel's file
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * i; }
    // false: this or another wait of the CTA ran out
    __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
        if (phase_done(bar(i), parity)) return true;
        const uint64_t t0 = globaltimer();
        for (;;) {
            if (phase_done(bar(i), parity)) return true;
            if (*abort) return false;
            if (globaltimer() - t0 > kWaitLimitNs) {
                *abort = 1;
                atomicOr(error, kErrTimeout);
                return false;
            }
        }
    }
    // Whether all lanes' waits were met; the warp is converged behind it. What follows a wait (elect, TMEM loads and stores,
    // arrivals) takes the whole warp, and a lane that had given up alone would leave the others waiting for it.
    static __device__ __forceinline__ bool met(bool ok) { return __all_sync(0xffffffffu, ok); }
    // by a converged warp, once for all its lanes
    __device__ __forceinline__ void arrive(int i) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar(i));
    }
};

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// rows of `cols` elements, `stride` apart, in boxes of box_rows x 128 bytes, swizzled
inline bool encode(CUtensorMap *map, CUtensorMapDataType type, int bytes, const void *at, int64_t cols, int64_t rows,
                   int64_t stride, int box_rows) {
    auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(rows > 1 ? stride : cols) * bytes};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / bytes), static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
    return enc(map, type, 2, const_cast<void *>(at), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool encode(CUtensorMap *map, const void *at, int64_t cols, int64_t rows, int64_t stride, int box_rows) {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, at, cols, rows, stride, box_rows);
}

}  // namespace tc
}  // namespace scan
}  // namespace kda
