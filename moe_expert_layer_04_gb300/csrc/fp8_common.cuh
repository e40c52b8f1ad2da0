// fp8_common.cuh -- helpers of the FP8 operators whose operands carry one fp32
// scale per block of 128.
//
// A block is 128 consecutive elements along the contraction (of a row: token
// rows, 1 x 128) or a 128 x 128 tile (weights); a short last block holds what
// is left.  With amax the block's largest magnitude, at least 2^-100:
//   s = fl(amax / 448),  r = fl(448 / amax),  code = E4M3(fl(v r))
// (nearest value, ties to even) and the element stands for s * E4M3(code).
// One division per block instead of one per element; the floor keeps r finite
// and the codes of an all-zero block zero.  A block with a NaN has scale NaN,
// one with an infinity (and no NaN) scale infinity and code NaN at the
// infinite elements, so neither passes for a number downstream.
// ("DeepSeek-V4昇腾训练支持：基于 CANN 平台的TorchTitan-NPU + AutoFuse 极简训练优化
// 实践", 性能结果与未来展望: FP8 low-precision compute; the page fixes no format.)
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;
constexpr float kFp8AmaxFloor = 7.888609052210118e-31f;   // 2^-100

__host__ __device__ inline int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

// Scale s and factor r of a block from the largest magnitude's fp32 bits (sign
// cleared; as integers NaN > infinity > every number, so an integer maximum
// over a block keeps a NaN).
struct Fp8Scale {
    float s, r;
};
__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits);
    const float m = a < kFp8AmaxFloor ? kFp8AmaxFloor : a;   // a NaN stays
    return {__fdiv_rn(m, kFp8Max), __fdiv_rn(kFp8Max, m)};
}

// Two values -> two E4M3 codes, `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Codes of the bf16 pair `w` times r.
__device__ __forceinline__ uint32_t e4m3x2_bf16(uint32_t w, float r) {
    return e4m3x2(bf16_lo(w) * r, bf16_hi(w) * r);
}

// h = silu(min(g, c)) * clamp(u, -c, c); a NaN in g or u stays a NaN.
__device__ __forceinline__ float swiglu_clamped_nan(float g, float u, float c) {
    const float a = g > c ? c : g;
    const float b = u > c ? c : (u < -c ? -c : u);
    return a * __fdividef(1.0f, 1.0f + __expf(-a)) * b;
}

// Four E4M3 codes -> two f16 pairs, exact, a NaN code to a NaN: two conversion
// instructions.  (To bf16 there is none: through fp32 it takes eight, and by
// moving bits ten on the integer pipe, 0.75 us of the SM for 32 KB, as long as they
// take to arrive.)
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(w & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
}

// Two f16 that bf16 holds (E4M3 values) -> bf16, exact.
__device__ __forceinline__ uint32_t f16x2_bf16x2(uint32_t w) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return pack_bf16x2(v.x, v.y);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A group's first row as the rows of the call allow it: offsets come from the device,
// where the host cannot check them, and nothing may be read or written past the rows.
__device__ __forceinline__ int row_offset(int o, int max_rows) { return min(max(o, 0), max_rows); }

// Contiguous bytes into shared memory (both 16-byte aligned, bytes a multiple of
// 16), counted on an mbarrier.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes,
                                          uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// A launch that may begin before the kernel ahead of it in the stream ends
// (programmatic dependent launch), which hides its latency; such a kernel touches
// nothing in memory before wait_for_kernels_ahead().  (few_experts_kernel alone works
// beside the kernel ahead, its own gate, through signals in the workspace, and waits for
// its end before it ends itself: every kernel launched so must, as the one behind it
// waits for no other.)
template <typename... P, typename... A>
inline moe_status launch_early(void (*kern)(P...), dim3 grid, int threads, int smem,
                               cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, P(args)...) != cudaSuccess) return MOE_ERR_CUDA;
    return cuda_status(cudaGetLastError());
}
__device__ __forceinline__ void wait_for_kernels_ahead() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_kernels_behind_begin() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace moe
