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

// Three E5M2 terms of two fp16 values: each term is the upper byte of what is left, sign, exponent and two
// mantissa bits of an fp16, so cutting it off and subtracting it are exact; the last one is rounded. Of
// the 11 significant bits the terms hold at least the first 9: a relative error of 2^-9 at the most.
// Codes are the bytes 1 and 3 of t[k].  (The conversion instruction rounds each term but runs at a quarter of
// these operations' rate: 2880 ns a tile against 1590 in the 128-row kernel.)
__device__ __forceinline__ void e5m2_terms(__half2 y, uint32_t (&t)[3]) {
    auto bits = [](const __half2& h) { return *reinterpret_cast<const uint32_t*>(&h); };
    auto half = [](uint32_t u) { return *reinterpret_cast<const __half2*>(&u); };
    t[0] = bits(y) & 0xff00ff00u;
    y = __hsub2(y, half(t[0]));
    t[1] = bits(y) & 0xff00ff00u;
    y = __hsub2(y, half(t[1]));
    t[2] = bits(y) + 0x00800080u;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Instruction descriptor of an 8-bit float MMA (kind::f8f6f4), fp32 accumulator, both operands
// K-major, M = 128, N a multiple of 16: D format F32 (bits 4-5 = 1), A and B formats in bits 7-9
// and 10-12 (0 = E4M3, 1 = E5M2), N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_f8(uint32_t a_fmt, uint32_t b_fmt, int N) {
    return (1u << 4) | (a_fmt << 7) | (b_fmt << 10) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

// Shared-memory operand descriptors in two words.  The upper one (stride between 8-row groups, version)
// is a constant of the operand and the lower one (address, distance of the 16-byte K chunks) moves with the
// address by its sixteenth, so an MMA costs its issuing thread an addition or two.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr >> 4) & 0x3fffu) | ((lbo >> 4) << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14); }

// D += A B, both operands in shared memory.
template <bool ACC>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n}\n" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}

// The same with A in tensor memory.
__device__ __forceinline__ void mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], b, %4, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The kernels of this cache are launched as programmatic dependents of whatever precedes them on the stream: their
// blocks may be scheduled while that runs, let the next kernel's be scheduled in turn, and wait here, before they
// read, write or allocate anything (tensor memory held while waiting could be what the grid before needs).  Every
// block waits, also one without work, so that a grid's end implies the end of the grids before it.  Calls that
// follow one another on a stream cost about 2 us less each.  What earlier grids may have written is then read with plain
// loads: one through the read-only path (__ldg) need not stay behind the wait.
__device__ __forceinline__ void follow_grid() {
    asm volatile("griddepcontrol.launch_dependents;\n griddepcontrol.wait;" ::: "memory");
}

// Launches a kernel so, with clusters of `cluster` blocks where that is above 1.
template <class... P, class... A>
inline cudaError_t launch_following(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, unsigned cluster, cudaStream_t st,
                                    const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
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
