/*
 * mxfp4.h -- MXFP4 W4A4 linear layer, C-ABI of libmxfp8.so.
 *
 * OCP Microscaling MXFP4: E2M1 elements with one E8M0 scale per 32 (the block
 * and scale of mxfp8.h with 4-bit elements; nvfp4.h is the other 4-bit format,
 * with 16-element blocks, UE4M3 scales and a global scale).
 *
 *   per 32-element block x: e = floor(log2(max|x|)) - 2 (2 is the exponent of
 *     E2M1's top binade), clamped to [-127, 127], -127 for an all-zero block;
 *     codes E2M1(x / 2^e), nearest, ties to even, saturating at 6.  A block
 *     holding Inf/NaN gets scale byte 0xFF and codes 7.
 *   Y[m, n] = BF16_RNE(sum_b 2^(sx[m,b] + sw[n,b]) sum_j qx[m,32b+j] qw[n,32b+j]
 *                      + F32(bias[n])), FP32 accumulation
 *
 * The GEMM runs the block-scaled 4-bit tensor-core kind (tcgen05.mma
 * kind::mxf4, 32-element E8M0 scales) with the packed codes and the scale
 * atoms as stored.  Few rows (decoding, M <= MXFP4_FEW_ROWS), and more rows
 * where Y has no more 128 x 128 tiles than the GPU has SMs, take a kernel of
 * their own that is bound by reading the weights; it may split K into up to 8
 * parts that are summed in a fixed order, so a call's result is reproducible, but
 * the number of parts depends on M and N.
 *
 * Layouts: codes [rows, K/2] bytes, two E2M1 codes per byte, element 2i in the
 * low nibble (sign bit 3, exponent bits 2:1, mantissa bit 0); scales in the
 * tensor-core layout of mxfp8.h (512-byte atoms of 128 rows x 4 blocks of 32).
 * Ownership, streams and errors as in mxfp8.h.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include "mxfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* M up to which the few-rows kernel is always taken. */
#define MXFP4_FEW_ROWS 128

/* Bytes of the scale array for rows x K (K % 32 == 0), 0 on bad arguments. */
size_t mxfp4_scale_bytes(int64_t rows, int64_t K);

/*
 * Quantize BF16 activations X [M, K] (row stride ldx >= K, ldx % 8 == 0, X
 * 16-byte aligned): codes [M, K/2] (8-byte aligned), scales
 * mxfp4_scale_bytes(M, K) bytes (4-byte aligned, padding 0).  K % 32 == 0.
 */
mxfp8_status mxfp4_quantize_bf16(const void *X, int64_t M, int64_t K, int64_t ldx, void *codes, void *scales,
                                 mxfp8_stream_t stream);

/* Weights: FP32 W [N, K] (row stride K), the same rule on the FP32 values. */
mxfp8_status mxfp4_quantize_weight_f32(const float *W, int64_t N, int64_t K, void *Wq, void *Wscale,
                                       mxfp8_stream_t stream);

/*
 * The GEMM and epilogue on quantized operands: Xq [M, K/2] and Wq [N, K/2]
 * packed codes with their scales (mxfp4_scale_bytes of [M, K] and [N, K]),
 * bias F16 [N] or NULL, Y BF16 [M, N] (written).  Requires K % 32 == 0,
 * N % 8 == 0, N > 0, M >= 0, every pointer 16-byte aligned.
 */
mxfp8_status mxfp4_gemm(const void *Xq, const void *Xscale, int64_t M, int64_t K, const void *Wq,
                        const void *Wscale, int64_t N, const void *bias, void *Y, mxfp8_stream_t stream);

/* Workspace bytes mxfp4_linear needs: the activation codes (rounded up to
 * 256 bytes) and their scales. */
size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t K);

/*
 * The whole layer: mxfp4_quantize_bf16 of X (row stride K) into `workspace`,
 * then mxfp4_gemm.  workspace: >= mxfp4_linear_workspace_bytes(M, K) bytes,
 * 256-byte aligned, overwritten.  Requirements as mxfp4_gemm.
 */
mxfp8_status mxfp4_linear(const void *X, int64_t M, int64_t K, const void *Wq, const void *Wscale, int64_t N,
                          const void *bias, void *Y, void *workspace, size_t ws_bytes, mxfp8_stream_t stream);

/*
 * As mxfp8_rmsnorm_quantize and mxfp8_gated_quantize (mxfp8.h), with the
 * result quantized to MXFP4: codes [M, K/2] (8-byte aligned), scales
 * mxfp4_scale_bytes(M, K) bytes (4-byte aligned).  K % 32 == 0, M >= 0
 * (norm: K <= MXFP8_NORM_MAX_K).
 */
mxfp8_status mxfp4_rmsnorm_quantize(const void *X, int64_t ldx, const void *residual, int64_t ldr,
                                    void *residual_out, int64_t ldh, const void *weight, int weight_dtype,
                                    float eps, int64_t M, int64_t K, void *codes, void *scales,
                                    mxfp8_stream_t stream);
mxfp8_status mxfp4_gated_quantize(const void *gate, int64_t ldg, const void *up, int64_t ldu, int act, int64_t M,
                                  int64_t K, void *codes, void *scales, mxfp8_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
