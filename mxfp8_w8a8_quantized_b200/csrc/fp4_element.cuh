/*
 * fp4_element.cuh -- per-element arithmetic of the 4-bit formats (E2M1 codes;
 * NVFP4: UE4M3 scale per 16 elements and a global scale, MXFP4: E8M0 scale
 * per 32), shared by the quantizers and the kernels that write these formats
 * as their output.
 */
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

namespace mx {

/* max(|a|, |b|) of each BF16 half (sign = xor of the signs; a NaN gives the
 * canonical NaN) */
__device__ __forceinline__ uint32_t nq_absmax_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

/* 8 values -> 4 bytes of E2M1 pairs (even element in the low nibble). */
__device__ __forceinline__ uint32_t nq_e2m1x8(float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                              float x7)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
        : "=r"(r)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3), "f"(x4), "f"(x5), "f"(x6), "f"(x7));
    return r;
}

/* The UE4M3 scale byte of a 16-element NVFP4 block, RN(amax * gs) saturated
 * at 448, with gs = RN(g / 6). */
__device__ __forceinline__ uint32_t nvfp4_scale_byte(float amax, float gs)
{
    return (uint32_t)__nv_cvt_float_to_fp8(amax * gs, __NV_SATFINITE, __NV_E4M3) & 0x7Fu;
}

/* RN(g / dec(sb)), the factor of the block's elements; 0 when the scale is 0. */
__device__ __forceinline__ float nvfp4_multiplier(uint32_t sb, float g)
{
    const __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)sb, __NV_E4M3);
    const float ds = __half2float(__half(hr));
    return ds > 0.0f ? __fdiv_rn(g, ds) : 0.0f;
}

/* The E8M0 scale byte of a 32-element MXFP4 block from the bits of its amax
 * (binary32, sign cleared): e = floor(log2 amax) - 2, 2 being the exponent of
 * E2M1's top binade, clamped at -127; 0xFF for a block holding Inf or NaN. */
__device__ __forceinline__ uint32_t mxfp4_scale_byte(uint32_t abits)
{
    const uint32_t ef = abits >> 23;
    if (ef >= 255u)
        return 0xFFu;
    return ef > 2u ? ef - 2u : 0u;
}

} // namespace mx
