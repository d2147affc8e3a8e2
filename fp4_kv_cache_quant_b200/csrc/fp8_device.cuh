// fp8_device.cuh -- number formats, the tcgen05 8-bit MMA and small helpers of
// the 8-bit paged cache (bdfp8.h).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/bdfp8.h"
#include "bdfp4_device.cuh"
#include "tc_ptx.cuh"

namespace bdfp4 {
namespace fp8 {

constexpr int kBlockTokens = 16;                 // tokens that share a scale
constexpr int kBlocksPerPage = kPageSlots / kBlockTokens;
constexpr int kScalePage = 2 * kBlocksPerPage;   // floats of kv_scales per (page, head)

template <int FMT>
struct Fmt8;
template <>
struct Fmt8<BDFP8_E4M3> {
    static constexpr float top = 448.0f;
    static constexpr uint32_t mma = 0;   // operand format field of the instruction descriptor
};
template <>
struct Fmt8<BDFP8_E5M2> {
    static constexpr float top = 57344.0f;
    static constexpr uint32_t mma = 1;
};

// Two fp32 values to 8-bit floats (nearest, ties to even, saturating): lo's code in bits 0..7.
template <int FMT>
__device__ __forceinline__ uint32_t f8x2(float lo, float hi) {
    uint16_t r;
    if constexpr (FMT == BDFP8_E4M3) asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Instruction descriptor of an 8-bit float MMA (kind::f8f6f4), fp32 accumulator, both operands
// K-major, M = 128, N a multiple of 16: D format F32 (bits 4-5 = 1), A and B formats in bits 7-9
// and 10-12 (0 = E4M3, 1 = E5M2), N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_f8(uint32_t a_fmt, uint32_t b_fmt, int N) {
    return (1u << 4) | (a_fmt << 7) | (b_fmt << 10) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Raises a kernel's dynamic shared memory limit once per device and kernel (each caller has its
// own flags); concurrent first calls repeat the same setting.
template <class Kernel>
inline cudaError_t allow_smem(Kernel* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace fp8
}  // namespace bdfp4
