/*
 * fused_capi.cu -- C-ABI entry points of the kernels that write the next
 * linear's quantized input (RMS norm, gated activation) in every format, and
 * of the MXFP4 layer: argument checks, then launches on the caller's stream.
 */
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "capi_util.cuh"
#include "fp8_rowwise.h"
#include "fused_quant.cuh"
#include "mxfp4.h"
#include "mxfp8.h"
#include "nvfp4.h"
#include "quant_out.cuh"

namespace mx {
int launch_gemm(const void *Xq, const void *Xs, int64_t M, int64_t K, const void *Wq, const void *Ws, int64_t N,
                const void *bias, void *Y, int epi, void *S, cudaStream_t stream, unsigned long long timeout_ns,
                cudaError_t *err, const float *gx, const float *gw);
int launch_mxfp4_skinny(const void *Xq, const void *Xs, int64_t M, int64_t K, const void *Wq, const void *Ws,
                        int64_t N, const void *bias, void *Y, cudaStream_t stream, unsigned long long timeout_ns,
                        cudaError_t *err);
cudaError_t launch_mxfp4_quantize(const void *X, bool f32_in, int64_t M, int64_t K, int64_t ldx, uint8_t *Q,
                                  uint8_t *S, cudaStream_t stream);
} // namespace mx

using namespace mx;

static_assert(MXFP8_NORM_MAX_K == FUSED_MAX_ROW && FP8RW_MAX_K == FUSED_MAX_ROW, "row limits of the fused kernels");
static_assert((int)MXFP8_DTYPE_BF16 == NORM_W_BF16 && (int)MXFP8_DTYPE_F16 == NORM_W_F16 &&
                  (int)MXFP8_DTYPE_F32 == NORM_W_F32, "weight types");

namespace {

cudaStream_t stream_of(mxfp8_stream_t s)
{
    return reinterpret_cast<cudaStream_t>(s);
}

/* Elements a row's blocks (or, per row, its 16-byte loads) come in. */
int64_t k_multiple(int fmt)
{
    return fmt == OUT_FP8RW ? 8 : fmt == OUT_NVFP4 ? 16 : 32;
}

mxfp8_status out_format(int layout, int *fmt)
{
    if (layout != MXFP8_SF_ROWMAJOR && layout != MXFP8_SF_TCGEN05)
        return MXFP8_ERR_ARG;
    *fmt = layout == MXFP8_SF_TCGEN05 ? OUT_MXFP8_TC : OUT_MXFP8_ROW;
    return MXFP8_OK;
}

/* A BF16 input or output of K columns: stride in elements, 16-byte rows. */
mxfp8_status rows_args(const void *p, int64_t ld, int64_t K)
{
    if (!p || ld < K)
        return MXFP8_ERR_ARG;
    return aligned(p, 16) && ld % 8 == 0 ? MXFP8_OK : MXFP8_ERR_ALIGN;
}

/* Checks shared by both kernels; fills o.  M > 0. */
mxfp8_status out_args(int fmt, int64_t M, int64_t K, int64_t max_k, const float *g, void *codes, void *scales,
                      QuantOut *o)
{
    if (!codes || !scales || (fmt == OUT_NVFP4 && !g))
        return MXFP8_ERR_ARG;
    if (K % k_multiple(fmt) != 0 || K > max_k || M > kMaxRows)
        return MXFP8_ERR_SHAPE;
    if (!aligned(codes, 8) || !aligned(scales, 4) || !aligned(g, 4))
        return MXFP8_ERR_ALIGN;
    const bool tc = fmt != OUT_MXFP8_ROW && fmt != OUT_FP8RW;
    o->Q = static_cast<uint8_t *>(codes);
    o->S = scales;
    o->g = g;
    o->K = (int)K;
    o->kg = (int)(fmt == OUT_NVFP4 ? (K + 63) / 64 : (K + 127) / 128);
    o->M = (int)M;
    o->rows = (int)(tc ? (M + 127) / 128 * 128 : M);
    return MXFP8_OK;
}

mxfp8_status rmsnorm_any(int fmt, const void *X, int64_t ldx, const void *residual, int64_t ldr, void *residual_out,
                         int64_t ldh, const void *weight, int weight_dtype, float eps, int64_t M, int64_t K,
                         const float *g, void *codes, void *scales, mxfp8_stream_t stream)
{
    if (M < 0 || K <= 0 || !(eps > 0.0f) || std::isinf(eps))
        return MXFP8_ERR_ARG;
    if (weight_dtype != MXFP8_DTYPE_BF16 && weight_dtype != MXFP8_DTYPE_F16 && weight_dtype != MXFP8_DTYPE_F32)
        return MXFP8_ERR_ARG;
    if (M == 0)
        return MXFP8_OK;
    if (!weight)
        return MXFP8_ERR_ARG;
    QuantOut o;
    mxfp8_status st = rows_args(X, ldx, K);
    if (st == MXFP8_OK && residual) {
        st = rows_args(residual, ldr, K);
        if (st == MXFP8_OK)
            st = rows_args(residual_out, ldh, K);
        /* in place only row by row */
        if (st == MXFP8_OK && ((residual_out == X && ldh != ldx) || (residual_out == residual && ldh != ldr)))
            st = MXFP8_ERR_ARG;
    }
    if (st == MXFP8_OK)
        st = out_args(fmt, M, K, MXFP8_NORM_MAX_K, g, codes, scales, &o);
    if (st == MXFP8_OK && !aligned(weight, 16))
        st = MXFP8_ERR_ALIGN;
    if (st != MXFP8_OK)
        return st;
    NormArgs p;
    p.x = static_cast<const uint16_t *>(X);
    p.r = static_cast<const uint16_t *>(residual);
    p.h = static_cast<uint16_t *>(residual_out);
    p.w = weight;
    p.wtype = weight_dtype;
    p.ldx = ldx;
    p.ldr = ldr;
    p.ldh = ldh;
    p.eps = eps;
    p.inv_k = 1.0 / (double)K;
    return from_cuda(launch_rmsnorm_quantize(fmt, p, o, stream_of(stream)));
}

mxfp8_status gated_any(int fmt, const void *gate, int64_t ldg, const void *up, int64_t ldu, int act, int64_t M,
                       int64_t K, const float *g, void *codes, void *scales, mxfp8_stream_t stream)
{
    if (M < 0 || K <= 0 || (act != MXFP8_ACT_SILU && act != MXFP8_ACT_GELU_TANH))
        return MXFP8_ERR_ARG;
    if (M == 0)
        return MXFP8_OK;
    QuantOut o;
    mxfp8_status st = rows_args(gate, ldg, K);
    if (st == MXFP8_OK)
        st = rows_args(up, ldu, K);
    if (st == MXFP8_OK)
        st = out_args(fmt, M, K, fmt == OUT_FP8RW ? FP8RW_MAX_K : kMaxK, g, codes, scales, &o);
    if (st != MXFP8_OK)
        return st;
    GatedArgs p;
    p.gate = static_cast<const uint16_t *>(gate);
    p.up = static_cast<const uint16_t *>(up);
    p.ldg = ldg;
    p.ldu = ldu;
    return from_cuda(launch_gated_quantize(fmt, act == MXFP8_ACT_GELU_TANH, p, o, stream_of(stream)));
}

mxfp8_status mxfp4_gemm_args(const void *Xq, const void *Xscale, int64_t M, int64_t K, const void *Wq,
                             const void *Wscale, int64_t N, const void *bias, const void *Y)
{
    if (M < 0 || K <= 0 || N <= 0)
        return MXFP8_ERR_ARG;
    if (M == 0)
        return MXFP8_OK;
    if (!Xq || !Xscale || !Wq || !Wscale || !Y)
        return MXFP8_ERR_ARG;
    if (K % 32 != 0 || N % 8 != 0 || M > kMaxRows || N > kMaxRows || K > kMaxK)
        return MXFP8_ERR_SHAPE;
    if (!aligned(Xq, 16) || !aligned(Xscale, 16) || !aligned(Wq, 16) || !aligned(Wscale, 16) || !aligned(Y, 16) ||
        (bias && !aligned(bias, 16)))
        return MXFP8_ERR_ALIGN;
    return MXFP8_OK;
}

mxfp8_status mxfp4_gemm_launch(const void *Xq, const void *Xscale, int64_t M, int64_t K, const void *Wq,
                               const void *Wscale, int64_t N, const void *bias, void *Y, mxfp8_stream_t stream)
{
    cudaError_t e;
    /* The few-rows kernel takes 128 x 128 tiles and can split K, the large one
     * 256 x 256 tiles on CTA pairs at twice the rate per operand byte.  Beyond
     * one tile of rows the former wins where its tiles fill no more than the
     * SMs, i.e. where the latter leaves most of them idle (K = N = 5120, M = 256:
     * 11.6 us against 14.5; M = 1021, 320 tiles: 23.7 against 21.4). */
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
    const int r = M <= MXFP4_FEW_ROWS || tiles <= device_sms()
                      ? launch_mxfp4_skinny(Xq, Xscale, M, K, Wq, Wscale, N, bias, Y, stream_of(stream), kWaitLimitNs,
                                            &e)
                      : launch_gemm(Xq, Xscale, M, K, Wq, Wscale, N, bias, Y, 5, nullptr, stream_of(stream),
                                    kWaitLimitNs, &e, nullptr, nullptr);
    if (r == 1)
        return MXFP8_ERR_CUDA; /* tensor map could not be encoded */
    return r == 0 ? MXFP8_OK : from_cuda(e);
}

} // namespace

extern "C" {

/* ------------------------------------------------------------ RMS norm */

mxfp8_status mxfp8_rmsnorm_quantize(const void *X, int64_t ldx, const void *residual, int64_t ldr,
                                    void *residual_out, int64_t ldh, const void *weight, int weight_dtype,
                                    float eps, int64_t M, int64_t K, void *codes, void *scales, int layout,
                                    mxfp8_stream_t stream)
{
    int fmt;
    const mxfp8_status st = out_format(layout, &fmt);
    if (st != MXFP8_OK)
        return st;
    return rmsnorm_any(fmt, X, ldx, residual, ldr, residual_out, ldh, weight, weight_dtype, eps, M, K, nullptr, codes,
                       scales, stream);
}

mxfp8_status fp8rw_rmsnorm_quantize(const void *X, int64_t ldx, const void *residual, int64_t ldr,
                                    void *residual_out, int64_t ldh, const void *weight, int weight_dtype,
                                    float eps, int64_t M, int64_t K, void *codes, float *scales,
                                    mxfp8_stream_t stream)
{
    return rmsnorm_any(OUT_FP8RW, X, ldx, residual, ldr, residual_out, ldh, weight, weight_dtype, eps, M, K, nullptr,
                       codes, scales, stream);
}

mxfp8_status nvfp4_rmsnorm_quantize(const void *X, int64_t ldx, const void *residual, int64_t ldr,
                                    void *residual_out, int64_t ldh, const void *weight, int weight_dtype,
                                    float eps, int64_t M, int64_t K, const float *global_scale, void *codes,
                                    void *scales, mxfp8_stream_t stream)
{
    return rmsnorm_any(OUT_NVFP4, X, ldx, residual, ldr, residual_out, ldh, weight, weight_dtype, eps, M, K,
                       global_scale, codes, scales, stream);
}

mxfp8_status mxfp4_rmsnorm_quantize(const void *X, int64_t ldx, const void *residual, int64_t ldr,
                                    void *residual_out, int64_t ldh, const void *weight, int weight_dtype,
                                    float eps, int64_t M, int64_t K, void *codes, void *scales,
                                    mxfp8_stream_t stream)
{
    return rmsnorm_any(OUT_MXFP4, X, ldx, residual, ldr, residual_out, ldh, weight, weight_dtype, eps, M, K, nullptr,
                       codes, scales, stream);
}

/* ---------------------------------------------------- gated activation */

mxfp8_status mxfp8_gated_quantize(const void *gate, int64_t ldg, const void *up, int64_t ldu, int act, int64_t M,
                                  int64_t K, void *codes, void *scales, int layout, mxfp8_stream_t stream)
{
    int fmt;
    const mxfp8_status st = out_format(layout, &fmt);
    if (st != MXFP8_OK)
        return st;
    return gated_any(fmt, gate, ldg, up, ldu, act, M, K, nullptr, codes, scales, stream);
}

mxfp8_status fp8rw_gated_quantize(const void *gate, int64_t ldg, const void *up, int64_t ldu, int act, int64_t M,
                                  int64_t K, void *codes, float *scales, mxfp8_stream_t stream)
{
    return gated_any(OUT_FP8RW, gate, ldg, up, ldu, act, M, K, nullptr, codes, scales, stream);
}

mxfp8_status nvfp4_gated_quantize(const void *gate, int64_t ldg, const void *up, int64_t ldu, int act, int64_t M,
                                  int64_t K, const float *global_scale, void *codes, void *scales,
                                  mxfp8_stream_t stream)
{
    return gated_any(OUT_NVFP4, gate, ldg, up, ldu, act, M, K, global_scale, codes, scales, stream);
}

mxfp8_status mxfp4_gated_quantize(const void *gate, int64_t ldg, const void *up, int64_t ldu, int act, int64_t M,
                                  int64_t K, void *codes, void *scales, mxfp8_stream_t stream)
{
    return gated_any(OUT_MXFP4, gate, ldg, up, ldu, act, M, K, nullptr, codes, scales, stream);
}

/* --------------------------------------------------------------- MXFP4 */

size_t mxfp4_scale_bytes(int64_t rows, int64_t K)
{
    return mxfp8_scale_bytes(rows, K, MXFP8_SF_TCGEN05);
}

static mxfp8_status mxfp4_quantize_any(const void *X, bool f32, int64_t M, int64_t K, int64_t ldx, void *codes,
                                       void *scales, mxfp8_stream_t stream)
{
    if (M < 0 || K <= 0 || ldx < K)
        return MXFP8_ERR_ARG;
    if (M == 0)
        return MXFP8_OK;
    if (!X || !codes || !scales)
        return MXFP8_ERR_ARG;
    if (K % 32 != 0 || M > kMaxRows || K > kMaxK)
        return MXFP8_ERR_SHAPE;
    if (!aligned(X, 16) || (ldx * (f32 ? 4 : 2)) % 16 != 0 || !aligned(codes, 8) || !aligned(scales, 4))
        return MXFP8_ERR_ALIGN;
    return from_cuda(launch_mxfp4_quantize(X, f32, M, K, ldx, static_cast<uint8_t *>(codes),
                                           static_cast<uint8_t *>(scales), stream_of(stream)));
}

mxfp8_status mxfp4_quantize_bf16(const void *X, int64_t M, int64_t K, int64_t ldx, void *codes, void *scales,
                                 mxfp8_stream_t stream)
{
    return mxfp4_quantize_any(X, false, M, K, ldx, codes, scales, stream);
}

mxfp8_status mxfp4_quantize_weight_f32(const float *W, int64_t N, int64_t K, void *Wq, void *Wscale,
                                       mxfp8_stream_t stream)
{
    return mxfp4_quantize_any(W, true, N, K, K, Wq, Wscale, stream);
}

mxfp8_status mxfp4_gemm(const void *Xq, const void *Xscale, int64_t M, int64_t K, const void *Wq,
                        const void *Wscale, int64_t N, const void *bias, void *Y, mxfp8_stream_t stream)
{
    const mxfp8_status st = mxfp4_gemm_args(Xq, Xscale, M, K, Wq, Wscale, N, bias, Y);
    if (st != MXFP8_OK || M == 0)
        return st;
    return mxfp4_gemm_launch(Xq, Xscale, M, K, Wq, Wscale, N, bias, Y, stream);
}

size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t K)
{
    if (M < 0 || K <= 0 || K % 32 != 0)
        return 0;
    return round_up((size_t)M * (size_t)(K / 2), 256) + mxfp4_scale_bytes(M, K);
}

mxfp8_status mxfp4_linear(const void *X, int64_t M, int64_t K, const void *Wq, const void *Wscale, int64_t N,
                          const void *bias, void *Y, void *workspace, size_t ws_bytes, mxfp8_stream_t stream)
{
    if (M < 0 || K <= 0 || N <= 0)
        return MXFP8_ERR_ARG;
    if (M == 0)
        return MXFP8_OK;
    if (!X || !workspace)
        return MXFP8_ERR_ARG;
    if (K % 32 != 0)
        return MXFP8_ERR_SHAPE;
    if (!aligned(workspace, 256) || !aligned(X, 16))
        return MXFP8_ERR_ALIGN;
    if (ws_bytes < mxfp4_linear_workspace_bytes(M, K))
        return MXFP8_ERR_ARG;
    uint8_t *codes = static_cast<uint8_t *>(workspace);
    uint8_t *scales = codes + round_up((size_t)M * (size_t)(K / 2), 256);
    /* every check of both steps before anything is launched */
    mxfp8_status st = mxfp4_gemm_args(codes, scales, M, K, Wq, Wscale, N, bias, Y);
    if (st != MXFP8_OK)
        return st;
    st = mxfp4_quantize_bf16(X, M, K, K, codes, scales, stream);
    if (st != MXFP8_OK)
        return st;
    return mxfp4_gemm_launch(codes, scales, M, K, Wq, Wscale, N, bias, Y, stream);
}

} // extern "C"
