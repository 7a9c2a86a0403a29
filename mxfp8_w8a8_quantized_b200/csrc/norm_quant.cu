/*
 * norm_quant.cu -- residual addition, root-mean-square norm and the
 * quantization of its result for the next linear, in one kernel (sm_100a).
 *
 *   h = BF16_RNE(x + r)                       (h = x without a residual)
 *   rstd = 1 / sqrt(sum_k h_k^2 / K + eps)
 *   t_k = h_k w_k,  y_k = t_k rstd            binary32
 *   codes, scales = the output format's quantization of y (no BF16 in between)
 *
 * The norm reads the residual stream as it is stored, so a later layer that
 * reads h sees the values that were normalized.  h is exact to one rounding:
 * the binary32 sum of two BF16 values is exact or far from a BF16 tie.
 * Squares are formed and summed in binary64, where no BF16 row overflows or
 * underflows, and rstd is applied as a pair of binary32 values, so that with a
 * BF16 or FP16 weight (t is exact) the one rounding that counts is that of y:
 * values next to a border between two codes then go to the side the formula has
 * them on.  (Above a root mean square of 2^100 the pair's lower part, above
 * 2^126 the upper one, too, becomes subnormal: y is then within 5 2^-24.)  The
 * binary64 sum costs 0 to 3 % against one in binary32 per thread (75348 x 5120
 * MXFP8 437 us against 433), 5 to 10 % without a residual (4099 x 5120 19.4 against
 * 18.4, 777 x 4128 5.2 against 4.7), and 0.2 us for one token; binary32 sums with a
 * second path for the rows that leave its range cost up to 9 %, with a second round
 * through the same code up to 6 % (and one rounding more).  Rounding is monotone, so
 * a row's largest |y| is what max|t| gives: the per-row scale of OUT_FP8RW needs no
 * second pass over the row.
 *
 * HBM-bound: 2 (x) + 2 (r) bytes read, 2 (h) + the codes written per element.
 * A row is a block's (128 to 512 threads, by its length) or, up to 1024
 * elements, a warp's; it stays in registers (packed BF16) between the sum of
 * squares and the codes, so it is read once.  A thread loads all of its 16-byte
 * chunks before it uses the first; several rows are resident per SM and hide
 * one another's block reduction (one barrier per row).
 *
 * Measured with a residual (us in a captured graph, and the fraction of the
 * measured copy rate): 75348 x 5120 MXFP8 437 (0.95), per-channel FP8 426
 * (0.97), MXFP4 412 (0.93), NVFP4 440 (0.88); 4099 x 5120 26.9 (0.84), 27.4
 * (0.82), 25.1 (0.83), 27.1 (0.78); 4096 x 16384 MXFP8 83 (0.87); 777 x 4128
 * 6.6; 1 x 5120 3.4, which is a launch and three dependent latencies.
 * While the kernel ahead ends, a block asks L2 for its first row and block 0 for
 * the weight, which the many weights of a decode step have pushed out of L2 by
 * then: 27.0 to 25.5 us at 4099 x 5120, 7.0 to 6.0 at 777 x 4128, and 1.1 us of
 * an MXFP4 feed-forward block at 1 to 16 rows (33.2 to 32.1), all measured with
 * the sums in binary32.
 * Copying the next row to shared memory while one is coded, as the gated
 * activation with per-row scales does, gained nothing at 5120 elements (4099
 * rows: 28.4 against 26.8), where seven rows per SM are resident anyway.
 */
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "async_copy.cuh"
#include "fused_quant.cuh"
#include "ptx.cuh"
#include "quant_out.cuh"

namespace mx {

/* Weights 8c .. 8c+7 of the norm as binary32 pairs.  Plain loads, not those of
 * the read-only path: the kernel ahead, with which this one overlaps, may have
 * written them (a norm whose weight another layer computes). */
__device__ __forceinline__ void load_weight8(const void *w, int type, int c, f32x2 (&o)[4])
{
    if (type == NORM_W_F32) {
        const uint4 a = static_cast<const uint4 *>(w)[2 * c];
        const uint4 b = static_cast<const uint4 *>(w)[2 * c + 1];
        o[0] = f2_pack(__uint_as_float(a.x), __uint_as_float(a.y));
        o[1] = f2_pack(__uint_as_float(a.z), __uint_as_float(a.w));
        o[2] = f2_pack(__uint_as_float(b.x), __uint_as_float(b.y));
        o[3] = f2_pack(__uint_as_float(b.z), __uint_as_float(b.w));
        return;
    }
    const uint4 v = static_cast<const uint4 *>(w)[c];
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (type == NORM_W_BF16) {
            o[i] = bf16x2_to_f32x2(u[i]);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            o[i] = f2_pack(f.x, f.y);
        }
    }
}

/* Sum of s and maximum of m over a warp. */
__device__ __forceinline__ void warp_sum_max(double &s, float &m)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        m = absmax_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    }
}

/* Blocks per SM, by which the registers are bounded.  Rows of up to 5120
 * elements: 7 (75348 x 5120 MXFP8 / per-channel FP8 / MXFP4 / NVFP4 437 / 426 /
 * 412 / 440 us; 6: 447 / 430 / 422 / 442, 8: 455 / 445 / 423 / 455); up to 2048
 * elements with half the chunks: 12 (16384 x 2048 41.4 / 43.9 / 39.3 / 42.6 us;
 * 7: 43.4 / 46.1 / 44.0 / 43.6.  Row-major MXFP8 scales, which spill there, 44.6
 * against 42.1: no GEMM reads that layout).  Longer rows: 1024 threads per SM
 * (4096 x 16384 per-channel FP8 80 us, 99 with one block, sums in binary32). */
constexpr int norm_blocks(int nt, int ch)
{
    return nt >= 256 ? 1024 / nt : ch <= 2 ? 12 : 7;
}

/*
 * TPR threads per row with CH chunks each, NT / TPR rows per block (a row is a
 * warp, which needs no block reduction, or the whole block).
 */
template <int FMT, int NT, int TPR, int CH>
__global__ void __launch_bounds__(NT, norm_blocks(NT, CH)) rmsnorm_quantize_kernel(const NormArgs p, const QuantOut o)
{
    grid_launch_dependents();
    {   /* the first row and, once, the weight, while the kernel ahead ends */
        const int64_t r = (int64_t)blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
        if (r < o.M && (threadIdx.x & 7) == 0)
#pragma unroll 1
            for (int c = threadIdx.x % TPR; c < o.K >> 3; c += TPR) {
                prefetch_l2(p.x + r * p.ldx + 8 * c);
                if (p.r)
                    prefetch_l2(p.r + r * p.ldr + 8 * c);
            }
        if (blockIdx.x == 0) {
            const int wbytes = o.K * (p.wtype == NORM_W_F32 ? 4 : 2);
#pragma unroll 1
            for (int i = threadIdx.x * 128; i < wbytes; i += NT * 128)
                prefetch_l2((const uint8_t *)p.w + i);
        }
    }
    grid_wait_ahead();
    __shared__ double rsum[2][NT / 32];
    __shared__ float rmax[2][NT / 32];
    constexpr int RPB = NT / TPR;
    static_assert(RPB == 1 || TPR == 32, "a row is a warp or a block");
    const int lane = threadIdx.x & 31;
    const int t = threadIdx.x % TPR;
    const int nchunks = o.K >> 3;
    const float g = FMT == OUT_NVFP4 ? *o.g : 1.0f;
    const float gs = __fdiv_rn(g, 6.0f);
    int it = 0;
    for (int64_t r64 = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; r64 < o.rows;
         r64 += (int64_t)gridDim.x * RPB, ++it) {
        const int r = (int)r64;
        if (r >= o.M) { /* uniform over the row's threads */
            zero_scale_row<FMT>(o, r, t, TPR);
            continue;
        }
        const uint4 *xr = reinterpret_cast<const uint4 *>(p.x + (int64_t)r * p.ldx);
        uint4 v[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = t + j * TPR;
            v[j] = c < nchunks ? __ldcs(xr + c) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (p.r) {
            const uint4 *rr = reinterpret_cast<const uint4 *>(p.r + (int64_t)r * p.ldr);
            uint4 *hr = reinterpret_cast<uint4 *>(p.h + (int64_t)r * p.ldh);
            uint4 u[CH];
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = t + j * TPR;
                u[j] = c < nchunks ? __ldcs(rr + c) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = t + j * TPR;
                v[j].x = f32x2_to_bf16x2(f2_add(bf16x2_to_f32x2(v[j].x), bf16x2_to_f32x2(u[j].x)));
                v[j].y = f32x2_to_bf16x2(f2_add(bf16x2_to_f32x2(v[j].y), bf16x2_to_f32x2(u[j].y)));
                v[j].z = f32x2_to_bf16x2(f2_add(bf16x2_to_f32x2(v[j].z), bf16x2_to_f32x2(u[j].z)));
                v[j].w = f32x2_to_bf16x2(f2_add(bf16x2_to_f32x2(v[j].w), bf16x2_to_f32x2(u[j].w)));
                if (c < nchunks)
                    hr[c] = v[j];
            }
        }
        double sum = 0.0;
        float tmax = 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const uint32_t w4[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a, b;
                f2_unpack(bf16x2_to_f32x2(w4[i]), a, b);
                sum = fma((double)a, (double)a, sum);
                sum = fma((double)b, (double)b, sum);
            }
            if constexpr (FMT == OUT_FP8RW) {
                const int c = t + j * TPR;
                if (c < nchunks) {
                    f32x2 w8[4];
                    load_weight8(p.w, p.wtype, c, w8);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w8[i] = f2_mul(bf16x2_to_f32x2(w4[i]), w8[i]);
                    tmax = absmax_nan(tmax, chunk_amax(w8));
                }
            }
        }
        warp_sum_max(sum, tmax);
        if constexpr (TPR > 32) {
            double *rs = rsum[it & 1]; /* alternate buffers: one barrier per row */
            float *rm = rmax[it & 1];
            if (lane == 0) {
                rs[threadIdx.x >> 5] = sum;
                rm[threadIdx.x >> 5] = tmax;
            }
            __syncthreads();
            sum = rs[0];
            tmax = rm[0];
#pragma unroll
            for (int w = 1; w < NT / 32; ++w) {
                sum += rs[w];
                tmax = absmax_nan(tmax, rm[w]);
            }
        }
        const double rstd = rsqrt(sum * p.inv_k + p.eps);
        const float rh = (float)rstd, rl = (float)(rstd - (double)rh);
        const f32x2 rh2 = f2_pack(rh, rh), rl2 = f2_pack(rl, rl);
        uint8_t *qrow = code_row<FMT>(o, r);
        uint8_t *srow = scale_row<FMT>(o, r);
        float sc = 0.0f, rcp = 0.0f;
        bool exact_row = false;
        if constexpr (FMT == OUT_FP8RW) {
            sc = __fdiv_rn(fmaf(tmax, rh, tmax * rl), 448.0f);
            rcp = __frcp_rn(sc);
            exact_row = rw_exact_row(sc, rcp);
            if (t == 0)
                static_cast<float *>(o.S)[r] = sc;
        }
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = t + j * TPR;
            if (c - lane >= nchunks) /* warp-uniform */
                break;
            const bool valid = c < nchunks;
            const uint32_t w4[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            f32x2 y[4] = {0ull, 0ull, 0ull, 0ull};
            if (valid) {
                load_weight8(p.w, p.wtype, c, y);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = f2_mul(bf16x2_to_f32x2(w4[i]), y[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = f2_fma(y[i], rh2, f2_mul(y[i], rl2));
            }
            if constexpr (FMT == OUT_FP8RW) {
                if (valid)
                    reinterpret_cast<uint2 *>(qrow)[c] = rw_chunk_codes(y, sc, rcp, exact_row);
            } else {
                store_chunk<FMT>(y, c, valid, lane, qrow, srow, o.kg, g, gs);
            }
        }
    }
}

template <int FMT, int NT, int TPR, int CH>
static cudaError_t launch_nt(const NormArgs &p, const QuantOut &o, cudaStream_t stream)
{
    constexpr int RPB = NT / TPR;
    int64_t blocks = ((int64_t)o.rows + RPB - 1) / RPB;
    const int64_t cap = (int64_t)device_sms() * (4096 / NT); /* several waves: fewer leave a longer last one */
    if (blocks > cap)
        blocks = cap;
    return launch_chained(rmsnorm_quantize_kernel<FMT, NT, TPR, CH>, dim3((unsigned)blocks), dim3(NT), 0, stream, 1, p,
                          o);
}

template <int FMT>
static cudaError_t launch_fmt(const NormArgs &p, const QuantOut &o, cudaStream_t stream)
{
    const int nchunks = o.K / 8;
    if (nchunks <= 128)
        return launch_nt<FMT, 128, 32, 4>(p, o, stream);
    if (nchunks <= 256)
        return launch_nt<FMT, 128, 128, 2>(p, o, stream);
    if (nchunks <= 640)
        return launch_nt<FMT, 128, 128, 5>(p, o, stream);
    if (nchunks <= 1024)
        return launch_nt<FMT, 256, 256, 4>(p, o, stream);
    return launch_nt<FMT, 512, 512, 4>(p, o, stream);
}

cudaError_t launch_rmsnorm_quantize(int fmt, const NormArgs &p, const QuantOut &o, cudaStream_t stream)
{
    if (o.rows == 0)
        return cudaSuccess;
    switch (fmt) {
    case OUT_MXFP8_TC:
        return launch_fmt<OUT_MXFP8_TC>(p, o, stream);
    case OUT_MXFP8_ROW:
        return launch_fmt<OUT_MXFP8_ROW>(p, o, stream);
    case OUT_FP8RW:
        return launch_fmt<OUT_FP8RW>(p, o, stream);
    case OUT_NVFP4:
        return launch_fmt<OUT_NVFP4>(p, o, stream);
    default:
        return launch_fmt<OUT_MXFP4>(p, o, stream);
    }
}

} // namespace mx
