/*
 * mxfp4_quant.cu -- MXFP4 quantization (sm_100a): packed E2M1 codes with one
 * E8M0 scale per 32 elements (OCP Microscaling Formats v1.0: the MXFP8 rule
 * of this library with E2M1's top exponent, 2, in the place of E4M3's 8).
 *
 * Per 32-element block: e = clamp(floor(log2 amax) - 2, -127); codes =
 * E2M1(x 2^-e), nearest even, saturating at 6 (a power-of-two multiply of a
 * BF16 or FP32 value is exact, so there is one rounding).  A block holding Inf
 * or NaN gets scale byte 0xFF and codes 7.  Codes are packed two per byte, the
 * even element in the low nibble; scales go into the tensor-core layout.
 *
 * HBM-bound: 2 (BF16) or 4 (FP32) bytes read, 1/2 + 1/32 byte written per
 * element.  A lane owns 16 elements (two or four 16-byte loads), two lanes a
 * block (one shuffle), eight lanes a 32-bit scale word.  A unit of work is a
 * row's 512-element segment; a warp walks whole rows when there are many, and
 * single segments when there are too few rows to fill the GPU, so that one
 * token's quantization is spread over all the warps it can use.  Measured:
 * 75348 x 5120 157 us, 0.94 of the copy rate; 4099 x 5120 10.8; 1021 x 4128 4.0 us;
 * 1 x 5120 1.6 us.  A warp asks L2 for its first segments while the kernel ahead
 * ends (without: 11.4, 4.5 and 1.7; linear of 33 x 13824 x 5120 13.5 -> 12.8 us).
 */
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "async_copy.cuh"
#include "fp4_element.cuh"
#include "fused_quant.cuh"
#include "mx_element.cuh"
#include "ptx.cuh"
#include "quant_out.cuh"

namespace mx {

constexpr int Q4_THREADS = 256;
constexpr int Q4_UNROLL = 2;

/* 16 consecutive elements as binary32 pairs */
template <bool F32_IN>
struct Q4Seg {
    uint4 v[F32_IN ? 4 : 2];
    __device__ __forceinline__ void load(const uint8_t *row, int k0)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(row + (int64_t)k0 * (F32_IN ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (F32_IN ? 4 : 2); ++i)
            v[i] = __ldcs(p + i);
    }
    __device__ __forceinline__ void pairs(f32x2 (&f)[8]) const
    {
        if constexpr (F32_IN) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = f2_pack(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
                f[2 * i + 1] = f2_pack(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[4 * i] = bf16x2_to_f32x2(v[i].x);
                f[4 * i + 1] = bf16x2_to_f32x2(v[i].y);
                f[4 * i + 2] = bf16x2_to_f32x2(v[i].z);
                f[4 * i + 3] = bf16x2_to_f32x2(v[i].w);
            }
        }
    }
    __device__ __forceinline__ float amax() const
    {
        if constexpr (F32_IN) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m = absmax_nan(m, __uint_as_float(v[i].x));
                m = absmax_nan(m, __uint_as_float(v[i].y));
                m = absmax_nan(m, __uint_as_float(v[i].z));
                m = absmax_nan(m, __uint_as_float(v[i].w));
            }
            return m;
        } else {
            const uint32_t a = nq_absmax_bf16x2(nq_absmax_bf16x2(v[0].x, v[0].y), nq_absmax_bf16x2(v[0].z, v[0].w));
            const uint32_t b = nq_absmax_bf16x2(nq_absmax_bf16x2(v[1].x, v[1].y), nq_absmax_bf16x2(v[1].z, v[1].w));
            const uint32_t m2 = nq_absmax_bf16x2(a, b) & 0x7FFF7FFFu;
            /* non-negative BF16 bit patterns order like their values */
            return __uint_as_float(max(m2 << 16, m2 & 0xFFFF0000u));
        }
    }
};

template <bool F32_IN>
__global__ void __launch_bounds__(Q4_THREADS) mxfp4_quantize_kernel(const void *X, int64_t ldx,
                                                                    const QuantOut o, int nseg, int spw)
{
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warp0 = ((int64_t)blockIdx.x * Q4_THREADS + threadIdx.x) >> 5;
    const int64_t nwarps = ((int64_t)gridDim.x * Q4_THREADS) >> 5;
    const int parts = (nseg + spw - 1) / spw; /* warps per row, spw segments each */
    const int64_t units = (int64_t)o.rows * parts;
    constexpr int EB = F32_IN ? 4 : 2;
    if (warp0 < units) { /* the first segments, while the kernel ahead ends */
        const int r = (int)(warp0 / parts);
        const int j0 = (int)(warp0 - (int64_t)r * parts) * spw;
        const uint8_t *xrow = reinterpret_cast<const uint8_t *>(X) + (int64_t)r * ldx * EB;
#pragma unroll
        for (int i = 0; i < Q4_UNROLL; ++i) {
            const int k0 = (j0 + i) * 512 + lane * 16;
            if (r < o.M && j0 + i < nseg && k0 < o.K && lane % (8 / EB) == 0)
                prefetch_l2(xrow + (int64_t)k0 * EB);
        }
    }
    grid_wait_ahead();

    for (int64_t t = warp0; t < units; t += nwarps) {
        const int r = (int)(t / parts);
        const int j0 = (int)(t - (int64_t)r * parts) * spw;
        const int j1 = min(j0 + spw, nseg);
        const bool row_ok = r < o.M;
        const uint8_t *xrow = reinterpret_cast<const uint8_t *>(X) + (int64_t)r * ldx * EB;
        uint8_t *qrow = o.Q + (int64_t)r * (o.K >> 1);
        uint8_t *srow = scale_row<OUT_MXFP4>(o, r);
        for (int j = j0; j < j1; j += Q4_UNROLL) {
            Q4Seg<F32_IN> seg[Q4_UNROLL];
            int k0[Q4_UNROLL];
            bool valid[Q4_UNROLL];
#pragma unroll
            for (int i = 0; i < Q4_UNROLL; ++i) {
                k0[i] = (j + i) * 512 + lane * 16;
                valid[i] = row_ok && j + i < j1 && k0[i] < o.K;
                if (valid[i])
                    seg[i].load(xrow, k0[i]);
            }
#pragma unroll
            for (int i = 0; i < Q4_UNROLL; ++i) {
                if (j + i >= j1) /* warp-uniform */
                    break;
                float amax = valid[i] ? seg[i].amax() : 0.0f;
                amax = absmax_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
                const uint32_t sb = valid[i] ? mxfp4_scale_byte(__float_as_uint(amax)) : 0u;
                if (valid[i]) {
                    f32x2 f[8];
                    seg[i].pairs(f);
                    const float m = inv_scale(sb);
                    const f32x2 mm = f2_pack(m, m);
                    float v[16];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        f2_unpack(f2_mul(f[k], mm), v[2 * k], v[2 * k + 1]);
                    uint2 q = make_uint2(nq_e2m1x8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]),
                                         nq_e2m1x8(v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]));
                    if (sb == 0xFFu)
                        q = make_uint2(0x77777777u, 0x77777777u);
                    *reinterpret_cast<uint2 *>(qrow + (k0[i] >> 1)) = q;
                }
                /* word of the four blocks that start at this lane's (8 lanes) */
                const uint32_t w = sb | (__shfl_down_sync(0xFFFFFFFFu, sb, 2) << 8) |
                                   (__shfl_down_sync(0xFFFFFFFFu, sb, 4) << 16) |
                                   (__shfl_down_sync(0xFFFFFFFFu, sb, 6) << 24);
                if ((lane & 7) == 0 && k0[i] < o.K)
                    *reinterpret_cast<uint32_t *>(srow + ((int64_t)(k0[i] >> 7) << 9)) = w;
            }
        }
    }
}

cudaError_t launch_mxfp4_quantize(const void *X, bool f32_in, int64_t M, int64_t K, int64_t ldx, uint8_t *Q,
                                  uint8_t *S, cudaStream_t stream)
{
    QuantOut o;
    o.Q = Q;
    o.S = S;
    o.g = nullptr;
    o.K = (int)K;
    o.kg = (int)((K + 127) / 128);
    o.M = (int)M;
    o.rows = (int)((M + 127) / 128 * 128);
    const int nseg = (int)((K + 511) / 512);
    if (o.rows == 0)
        return cudaSuccess;
    const int64_t cap = (int64_t)device_sms() * 8 * 4; /* 8 resident blocks x 4 waves */
    /* whole rows per warp when the rows alone fill the GPU's warps once */
    const int spw = o.rows >= device_sms() * 64 ? nseg : Q4_UNROLL;
    const int64_t units = (int64_t)o.rows * ((nseg + spw - 1) / spw);
    int64_t blocks = (units + Q4_THREADS / 32 - 1) / (Q4_THREADS / 32);
    if (blocks > cap)
        blocks = cap;
    return launch_chained(f32_in ? mxfp4_quantize_kernel<true> : mxfp4_quantize_kernel<false>, dim3((unsigned)blocks),
                          dim3(Q4_THREADS), 0, stream, 1, X, ldx, o, nseg, spw);
}

} // namespace mx
