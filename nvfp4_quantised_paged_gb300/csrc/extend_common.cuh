// extend_common.cuh -- helpers of the two chunk-attention kernels (extend_attention.cu, latent_extend.cu).
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace nvfp4kv {

namespace {

constexpr uint32_t kWaitLimitE = 1u << 24;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}


// Bounded wait on an mbarrier phase without sleeping between polls (these
// waits are on the critical path); gives up when another warp has aborted.
__device__ __forceinline__ bool spin_wait(uint64_t *bar, uint32_t parity, const volatile int *abort_flag) {
    for (uint32_t n = 0; n < kWaitLimitE; n++) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
    }
    return false;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// (a.x * b + c, a.y * b + c) in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
    uint64_t d;
    const uint64_t bb = (uint64_t)__float_as_uint(b) | ((uint64_t)__float_as_uint(b) << 32);
    const uint64_t cc = (uint64_t)__float_as_uint(c) | ((uint64_t)__float_as_uint(c) << 32);
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"((uint64_t)__float_as_uint(a.x) | ((uint64_t)__float_as_uint(a.y) << 32)), "l"(bb), "l"(cc));
    return make_float2(__uint_as_float((uint32_t)d), __uint_as_float((uint32_t)(d >> 32)));
}

// s0 += low BF16 of w, s1 += high BF16 of w (exact products by 1.0, FP32 sums)
__device__ __forceinline__ void add_bf16x2(float &s0, float &s1, uint32_t w) {
    const unsigned short one = 0x3f80;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2;\n"
        "fma.rn.f32.bf16 %0, lo, %3, %0; fma.rn.f32.bf16 %1, hi, %3, %1; }"
        : "+f"(s0), "+f"(s1)
        : "r"(w), "h"(one));
}

// cuTensorMapEncodeTiled, resolved from the driver once (a second thread waits for the first).
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(p);
        return nullptr;
    }();
    return fn;
}

}  // namespace

}  // namespace nvfp4kv
