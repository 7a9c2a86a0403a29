/*
 * rw_element.cuh -- per-element arithmetic of the per-channel FP8 format
 * (scale s = amax / 448, codes E4M3(x / s)), shared by the stand-alone
 * quantizer and the kernels that write this format as their output.
 */
#pragma once

#include <cuda_fp8.h>
#include <cstdint>

#include "mx_element.cuh"

namespace mx {

/*
 * RN(a / s) for a pair of binary32 values, given r = RN(1 / s), without a
 * division (Markstein's correction step with a fused multiply-add:
 * P. Markstein, "Computation of elementary functions on the IBM RISC
 * System/6000 processor", IBM J. Res. Dev. 34(1), 1990): q0 = RN(a r) is
 * within an ulp of a / s, so the residual a - q0 s is exact in one FMA, and
 * RN(q0 + (a - q0 s) r) is the correctly rounded quotient.  The step fails
 * for divisors whose significand is all ones; rows with such a scale (and
 * rows whose reciprocal overflows, or whose scale is 0) divide instead (see
 * rw_exact_row).  ns2 holds -s.
 */
__device__ __forceinline__ f32x2 rw_quot2(f32x2 a, f32x2 r2, f32x2 ns2)
{
    const f32x2 q0 = f2_mul(a, r2);
    return f2_fma(f2_fma(q0, ns2, a), r2, q0);
}

/* Rows whose codes take the plain division: 1/s not a positive finite value (s =
 * 0, i.e. all +-0, or so small that 1/s overflows, Inf, NaN), or a significand at
 * or near all ones. */
__device__ __forceinline__ bool rw_exact_row(float s, float rcp)
{
    return !(rcp > 0.0f && rcp < 3.0e38f) || (__float_as_uint(s) & 0x7FFFFFu) >= 0x7FFFF0u;
}

__device__ __forceinline__ uint32_t rw_e4m3x2(float lo, float hi)
{
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

/* Codes of the two BF16 values of a word (low half first), 16 bits. */
__device__ __forceinline__ uint32_t rw_codes_bf16x2(uint32_t w, f32x2 r2, f32x2 ns2)
{
    float lo, hi;
    f2_unpack(rw_quot2(bf16x2_to_f32x2(w), r2, ns2), lo, hi);
    return rw_e4m3x2(lo, hi);
}

/* The same by plain division (rows of rw_exact_row); s = 0 keeps x (+-0). */
__device__ __forceinline__ uint32_t rw_codes2_div(float a, float b, float s)
{
    return s == 0.0f ? rw_e4m3x2(a, b) : rw_e4m3x2(__fdiv_rn(a, s), __fdiv_rn(b, s));
}

} // namespace mx
