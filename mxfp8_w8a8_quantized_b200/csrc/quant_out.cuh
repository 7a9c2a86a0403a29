/*
 * quant_out.cuh -- writes a row of binary32 values as the quantized input of
 * the next linear, in any of the library's formats, from the registers of
 * the kernel that computed them.
 *
 * The unit is a chunk: 8 consecutive elements of a row per lane, so a warp
 * covers 256 consecutive elements, i.e. 8 blocks of 32 (4 lanes each) or 16
 * blocks of 16 (2 lanes each).  Block maxima and the scale words of the
 * tensor-core layout (four consecutive blocks of a row, one 32-bit word) are
 * combined by shuffles inside the warp; codes leave as one 8-byte (E4M3) or
 * 4-byte (E2M1) store per lane.  The values are quantized as they are, in
 * binary32: there is no rounding to BF16 in between.
 */
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "fp4_element.cuh"
#include "mx_element.cuh"
#include "rw_element.cuh"

namespace mx {

enum OutFmt : int {
    OUT_MXFP8_TC = 0,  /* E4M3, E8M0 per 32 in the tensor-core layout */
    OUT_MXFP8_ROW = 1, /* E4M3, E8M0 per 32, row-major */
    OUT_FP8RW = 2,     /* E4M3, FP32 scale per row */
    OUT_NVFP4 = 3,     /* E2M1, UE4M3 per 16, tensor-core layout, global scale */
    OUT_MXFP4 = 4,     /* E2M1, E8M0 per 32, tensor-core layout */
};

/* Output arrays of a quantizing kernel. */
struct QuantOut {
    uint8_t *Q;     /* codes */
    void *S;        /* scales: bytes, or one float per row (OUT_FP8RW) */
    const float *g; /* global scale (OUT_NVFP4) */
    int K;          /* elements per row */
    int kg;         /* 512-byte scale atoms per 128 rows (tensor-core layouts) */
    int M;          /* rows */
    int rows;       /* rows that own scale bytes: M, or M rounded up to 128 */
};

template <int FMT>
constexpr bool fmt_tc = FMT == OUT_MXFP8_TC || FMT == OUT_NVFP4 || FMT == OUT_MXFP4;
template <int FMT>
constexpr bool fmt_fp4 = FMT == OUT_NVFP4 || FMT == OUT_MXFP4;

/* First code byte of row r. */
template <int FMT>
__device__ __forceinline__ uint8_t *code_row(const QuantOut &o, int r)
{
    return o.Q + (int64_t)r * (fmt_fp4<FMT> ? o.K >> 1 : o.K);
}

/* Scale word 0 of row r in the tensor-core layout (word i is 512 i bytes
 * on), or the first scale byte of the row. */
template <int FMT>
__device__ __forceinline__ uint8_t *scale_row(const QuantOut &o, int r)
{
    uint8_t *S = static_cast<uint8_t *>(o.S);
    if constexpr (fmt_tc<FMT>)
        return S + (((int64_t)(r >> 7) * o.kg) << 9) + ((r & 31) << 4) + (((r >> 5) & 3) << 2);
    else
        return S + (int64_t)r * (o.K >> 5);
}

/* max(a, |b|) with NaN kept (a >= 0 or NaN). */
__device__ __forceinline__ float absmax_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

/* max(|a|, |b|, |c|), NaN if any of them is. */
__device__ __forceinline__ float absmax3_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

/* Largest magnitude of a chunk (NaN if any element is). */
__device__ __forceinline__ float chunk_amax(const f32x2 (&y)[4])
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f2_unpack(y[i], v[2 * i], v[2 * i + 1]);
    return absmax3_nan(absmax3_nan(v[0], v[1], v[2]), absmax3_nan(v[3], v[4], v[5]), absmax_nan(fabsf(v[6]), v[7]));
}

__device__ __forceinline__ void f2_unpack4(const f32x2 (&y)[4], f32x2 mul, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f2_unpack(f2_mul(y[i], mul), v[2 * i], v[2 * i + 1]);
}

/*
 * Quantizes chunk c (elements 8c .. 8c+7) of a row whose blocks scale on
 * their own (every format but OUT_FP8RW) and stores codes and scales.  All
 * 32 lanes call it, on chunks c0 + lane with c0 a multiple of 32; `valid` is
 * false for lanes past the row's end, which write no codes and, up to the end
 * of the last scale atom, zero scales.  The first lane of a block stores its
 * scale byte: one store instruction per warp and chunk, where gathering words
 * by shuffles took six more.  g, gs: the global scale and RN(g / 6) (OUT_NVFP4).
 */
template <int FMT>
__device__ __forceinline__ void store_chunk(const f32x2 (&y)[4], int c, bool valid, int lane, uint8_t *qrow,
                                            uint8_t *srow, int kg, float g, float gs)
{
    static_assert(FMT != OUT_FP8RW, "per-row scales are not per block");
    constexpr int LPB = FMT == OUT_NVFP4 ? 2 : 4; /* lanes per block */
    float amax = chunk_amax(y);
    amax = absmax_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    if constexpr (LPB == 4)
        amax = absmax_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    uint32_t sb;
    if constexpr (FMT == OUT_NVFP4) {
        sb = nvfp4_scale_byte(amax, gs);
        const float mul = nvfp4_multiplier(sb, g);
        float v[8];
        f2_unpack4(y, f2_pack(mul, mul), v);
        const uint32_t q = nq_e2m1x8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
        if (valid)
            reinterpret_cast<uint32_t *>(qrow)[c] = q;
    } else if constexpr (FMT == OUT_MXFP4) {
        sb = mxfp4_scale_byte(__float_as_uint(amax));
        const float mul = inv_scale(sb);
        float v[8];
        f2_unpack4(y, f2_pack(mul, mul), v);
        const uint32_t q = nq_e2m1x8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
        if (valid)
            reinterpret_cast<uint32_t *>(qrow)[c] = sb == 0xFFu ? 0x77777777u : q;
    } else {
        sb = scale_byte_from_amax(__float_as_uint(amax));
        const float mul = inv_scale(sb);
        float v[8];
        f2_unpack4(y, f2_pack(mul, mul), v);
        uint2 q = make_uint2(pack4_e4m3(v[0], v[1], v[2], v[3]), pack4_e4m3(v[4], v[5], v[6], v[7]));
        if (sb == 0xFFu)
            q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        if (valid)
            reinterpret_cast<uint2 *>(qrow)[c] = q;
    }
    if constexpr (fmt_tc<FMT>) {
        constexpr int LPA = 4 * LPB; /* chunks per scale atom of a row */
        if ((lane & (LPB - 1)) == 0 && c < kg * LPA)
            srow[((int64_t)(c / LPA) << 9) + (c % LPA) / LPB] = valid ? (uint8_t)sb : (uint8_t)0;
    } else {
        if (valid && (lane & 3) == 0)
            srow[c >> 2] = (uint8_t)sb;
    }
}

/* Codes of a chunk of a row with scale s (OUT_FP8RW); rcp = RN(1 / s),
 * exact_row = rw_exact_row(s, rcp). */
__device__ __forceinline__ uint2 rw_chunk_codes(const f32x2 (&y)[4], float s, float rcp, bool exact_row)
{
    uint32_t o[4];
    if (!exact_row) {
        const f32x2 r2 = f2_pack(rcp, rcp), ns2 = f2_pack(-s, -s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2_unpack(rw_quot2(y[i], r2, ns2), a, b);
            o[i] = rw_e4m3x2(a, b);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2_unpack(y[i], a, b);
            o[i] = rw_codes2_div(a, b, s);
        }
    }
    return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

/* Zero scale words of a padding row (rows [M, rows) of the tensor-core
 * layouts), by `n` threads of which this is number t. */
template <int FMT>
__device__ __forceinline__ void zero_scale_row(const QuantOut &o, int r, int t, int n)
{
    if constexpr (fmt_tc<FMT>) {
        uint8_t *srow = scale_row<FMT>(o, r);
        for (int i = t; i < o.kg; i += n)
            *reinterpret_cast<uint32_t *>(srow + ((int64_t)i << 9)) = 0u;
    }
}

} // namespace mx
