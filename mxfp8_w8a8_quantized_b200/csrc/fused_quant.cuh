/*
 * fused_quant.cuh -- arguments and launchers of the kernels that write the
 * next linear's quantized input: the RMS norm and the gated activation.
 */
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace mx {

struct QuantOut;

/* Types of the norm's weight (mxfp8_dtype of the C-ABI). */
enum NormWeight : int { NORM_W_BF16 = 0, NORM_W_F16 = 1, NORM_W_F32 = 2 };

/* Longest row of the norm and of the per-row-scaled gated activation. */
constexpr int FUSED_MAX_ROW = 16384;

struct NormArgs {
    const uint16_t *x; /* BF16 rows, ldx elements apart */
    const uint16_t *r; /* residual (BF16) or null */
    uint16_t *h;       /* x + r; may be x's or r's own memory */
    const void *w;     /* [K] */
    int wtype;
    int64_t ldx, ldr, ldh;
    float eps;
};

struct GatedArgs {
    const uint16_t *gate, *up; /* BF16 rows */
    int64_t ldg, ldu;
};

cudaError_t launch_rmsnorm_quantize(int fmt, const NormArgs &p, const QuantOut &o, cudaStream_t stream);
cudaError_t launch_gated_quantize(int fmt, bool gelu, const GatedArgs &p, const QuantOut &o, cudaStream_t stream);

/* SM count of the current device (148 if it cannot be read). */
int device_sms();

} // namespace mx
