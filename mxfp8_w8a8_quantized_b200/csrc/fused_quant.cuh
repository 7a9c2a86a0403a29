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
    double eps, inv_k; /* inv_k = 1 / K */
};

struct GatedArgs {
    const uint16_t *gate, *up; /* BF16 rows */
    int64_t ldg, ldu;
};

cudaError_t launch_rmsnorm_quantize(int fmt, const NormArgs &p, const QuantOut &o, cudaStream_t stream);
cudaError_t launch_gated_quantize(int fmt, bool gelu, const GatedArgs &p, const QuantOut &o, cudaStream_t stream);

/* SM count of the current device (148 if it cannot be read). */
int device_sms();

/*
 * Launches a kernel of this library with programmatic serialization: it may
 * start while the kernel ahead on the stream still runs, once every block of
 * that one has called grid_launch_dependents() (or ended).  Such a kernel
 * touches no global memory before grid_wait_ahead(), except for prefetches
 * into L2, which is where all SMs' writes meet; so nothing depends on what the
 * kernel ahead is.  cluster: blocks per cluster along x.
 */
template <class... P, class... A>
static inline cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                         int cluster, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

} // namespace mx
