/*
 * gated_quant.cu -- the gated activation of a feed-forward block and the
 * quantization of its result for the down projection, in one kernel
 * (sm_100a).
 *
 *   y = act(g) u,  act = SiLU: g / (1 + e^-g), or GELU in its tanh form:
 *                  g / (1 + e^-2v), v = sqrt(2/pi) (g + 0.044715 g^3)
 *   codes, scales = the output format's quantization of y
 *
 * everything in binary32, with no rounding to BF16 in between.  g and u are
 * row-strided views, usually the two halves of a fused projection's output.
 *
 * HBM-bound: 4 bytes read and the codes written per element; the two hardware
 * functions and some 17 further instructions per element come close to the
 * issue rate, so they are counted (packed binary32 pairs, three-input maxima, no
 * select and at most one clamp per gate).
 *  - Block-scaled formats: a thread owns one chunk of 8 columns and walks
 *    down the rows, so its addresses advance by constants; the next row's loads
 *    are in flight while a row is coded.  32760 x 13824 MXFP8: 398 to 424 us by
 *    the GPU, 0.82 to 0.87 of the measured copy rate (both activations), MXFP4 375
 *    (0.83), NVFP4 398 (0.79); 2047 x 13824: 25.0 to 25.8, 25.5, 26.0 us; 7 x
 *    13824: 2.1, NVFP4 2.6 us.  A thread asks L2 for its first row while the kernel
 *    ahead ends: 2.5 to 2.1 us at 7 rows, 6.5 to 6.2 at 300 (24.75 to 25.0 at 2047).
 *    With per-row scales, where the copies start at once, that gained nothing.
 *  - Per-row scales: one block (or warp) per row keeps the row's y in registers
 *    (binary32) until the row's maximum is known, so g and u are read once; each
 *    thread copies its part of the next row to shared memory meanwhile.  32760 x
 *    13824: 360 to 372 us, 0.93 to 0.96 of the copy rate (434 with plain loads);
 *    2047 x 13824: 27.1 to 27.8 us.
 */
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "async_copy.cuh"
#include "fused_quant.cuh"
#include "ptx.cuh"
#include "quant_out.cuh"

namespace mx {

/*
 * act(g) u of a pair: act(g) = g / (1 + e^-z) with z = g (SiLU) or 2v (GELU),
 * e^-z = 2^(-z log2 e) by the hardware exponential (relative error 2^-22).
 *
 * SiLU: g has 8 significant bits, so with log2 e cut to 16 bits (Lh) the
 * exponent -g Lh is exact in binary32; what Lh leaves out, Ll = 7.05e-6, comes in
 * as the factor 1 - g Ll ln 2 (|g| <= 88 matters: the square of that term is
 * below 2^-22), which the FMA that forms 1 + e^-z takes for free.  GELU: the
 * exponent is a polynomial whose roundings are larger than its own.
 *
 * Far below zero the exponential overflows and its reciprocal is 0; where that
 * reciprocal is below 2^-126 it flushes to 0 as well (act(g) is then below 1e-36
 * in magnitude).  NaN and +-Inf come out as the formula has them: the factor g
 * carries NaN and +Inf (SiLU's exponent takes no more than g = 256, so that its
 * correction stays finite), and -Inf times 0 is NaN.
 */
template <bool GELU>
__device__ __forceinline__ f32x2 gated2(uint32_t gw, uint32_t uw)
{
    const f32x2 g = bf16x2_to_f32x2(gw), u = bf16x2_to_f32x2(uw);
    const f32x2 one = f2_pack(1.0f, 1.0f);
    float t0, t1, d0, d1;
    if constexpr (GELU) {
        const float C1 = -2.302208185195923f;   /* -2 sqrt(2/pi) log2(e) */
        const float C3 = -0.10294324159622192f; /* -2 sqrt(2/pi) 0.044715 log2(e) */
        f2_unpack(f2_mul(g, f2_fma(f2_mul(g, g), f2_pack(C3, C3), f2_pack(C1, C1))), t0, t1);
        f2_unpack(f2_add(f2_pack(exp2_approx_ftz(t0), exp2_approx_ftz(t1)), one), d0, d1);
    } else {
        const float LH = 1.44268798828125f;         /* log2(e) cut to 16 bits */
        const float LL = 4.888495152129525e-06f;    /* (log2(e) - LH) ln 2 */
        float g0, g1;
        f2_unpack(g, g0, g1);
        const f32x2 z = f2_pack(fminf(g0, 256.0f), fminf(g1, 256.0f));
        f2_unpack(f2_mul(z, f2_pack(-LH, -LH)), t0, t1);
        f2_unpack(f2_fma(f2_pack(exp2_approx_ftz(t0), exp2_approx_ftz(t1)), f2_fma(z, f2_pack(-LL, -LL), one), one),
                  d0, d1);
    }
    return f2_mul(f2_mul(g, f2_pack(rcp_approx_ftz(d0), rcp_approx_ftz(d1))), u);
}

template <bool GELU>
__device__ __forceinline__ void gated_chunk(const uint4 &g, const uint4 &u, f32x2 (&y)[4])
{
    y[0] = gated2<GELU>(g.x, u.x);
    y[1] = gated2<GELU>(g.y, u.y);
    y[2] = gated2<GELU>(g.z, u.z);
    y[3] = gated2<GELU>(g.w, u.w);
}

constexpr int GT = 256;     /* threads per block */
constexpr int GAHEAD = 1;   /* rows loaded ahead of the one being coded */
/* Blocks per SM, by which the registers are bounded and the grid is counted
 * (NVFP4's second division needs the registers of 4). */
constexpr int gated_blocks(int fmt)
{
    return fmt == OUT_NVFP4 ? 4 : 5;
}

/*
 * Block-scaled formats.  A block is wx x wy warps: wx along the columns (256
 * each), wy along the rows; wx wy = 8, wx the power of two that reaches over the
 * row's segments (warps past the row's end return at once), or 8.
 */
template <int FMT, bool GELU>
__global__ void __launch_bounds__(GT, gated_blocks(FMT))
    gated_quantize_kernel(const GatedArgs p, const QuantOut o, int wx)
{
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wy = (GT / 32) / wx;
    const int nchunks = o.K >> 3;
    const int c0 = ((int)blockIdx.x * wx + warp % wx) * 32;
    const int c = c0 + lane;
    const bool col_ok = c < nchunks;
    {   /* the first row, while the kernel ahead ends */
        const int64_t r = (int64_t)blockIdx.y * wy + warp / wx;
        if (col_ok && r < o.M && (lane & 7) == 0) {
            prefetch_l2(p.gate + r * p.ldg + 8 * c);
            prefetch_l2(p.up + r * p.ldu + 8 * c);
        }
    }
    grid_wait_ahead();
    if (c0 >= nchunks)
        return;
    const float g = FMT == OUT_NVFP4 ? *o.g : 1.0f;
    const float gs = __fdiv_rn(g, 6.0f);
    const int step = (int)gridDim.y * wy;
    const int first = (int)blockIdx.y * wy + warp / wx;
    const uint4 *gp = reinterpret_cast<const uint4 *>(p.gate + (int64_t)first * p.ldg) + c;
    const uint4 *up = reinterpret_cast<const uint4 *>(p.up + (int64_t)first * p.ldu) + c;
    const int64_t gstep = (int64_t)step * (p.ldg >> 3), ustep = (int64_t)step * (p.ldu >> 3);
    int64_t rl = first; /* next row to load */
    uint4 gv[GAHEAD + 1], uv[GAHEAD + 1];
    auto load = [&](int i) {
        gv[i] = uv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (col_ok && rl < o.M) {
            gv[i] = __ldcs(gp);
            uv[i] = __ldcs(up);
        }
        gp += gstep;
        up += ustep;
        rl += step;
    };
#pragma unroll
    for (int i = 0; i < GAHEAD; ++i)
        load(i);
    for (int64_t r = first; r < o.rows; r += step) {
        load(GAHEAD);
        if (r < o.M) { /* warp-uniform */
            f32x2 y[4];
            gated_chunk<GELU>(gv[0], uv[0], y);
            store_chunk<FMT>(y, c, col_ok, lane, code_row<FMT>(o, (int)r), scale_row<FMT>(o, (int)r), o.kg, g, gs);
        } else if constexpr (fmt_tc<FMT>) {
            constexpr int LPA = FMT == OUT_NVFP4 ? 8 : 16; /* chunks per scale word */
            if (col_ok && (lane & (LPA - 1)) == 0)
                *reinterpret_cast<uint32_t *>(scale_row<FMT>(o, (int)r) + ((int64_t)(c / LPA) << 9)) = 0u;
        }
#pragma unroll
        for (int i = 0; i < GAHEAD; ++i) {
            gv[i] = gv[i + 1];
            uv[i] = uv[i + 1];
        }
    }
}

/* Per-row scales: TPR threads per row with CH chunks each, NT / TPR rows per
 * block; a row of one warp needs no block reduction. */
template <bool GELU, int NT, int TPR, int CH>
__global__ void __launch_bounds__(NT) gated_quantize_rowwise_kernel(const GatedArgs p, const QuantOut o)
{
    grid_launch_dependents();
    grid_wait_ahead();
    __shared__ float red[2][NT / 32];
    constexpr int RPB = NT / TPR; /* rows per block */
    static_assert(RPB == 1 || TPR == 32, "a row is a warp or a block");
    const int nchunks = o.K >> 3;
    const int t = threadIdx.x % TPR;
    /* this thread's chunks of a row: slot [j][gate / up][row of the block][t] */
    extern __shared__ uint4 ring[];
    uint4 *slot = ring + threadIdx.x;
    auto fetch = [&](int64_t r) {
        if (r >= o.M)
            return;
        const uint4 *gr = reinterpret_cast<const uint4 *>(p.gate + r * p.ldg);
        const uint4 *ur = reinterpret_cast<const uint4 *>(p.up + r * p.ldu);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = t + j * TPR;
            if (c < nchunks) {
                copy16_async(smem_u32(slot + 2 * j * NT), gr + c);
                copy16_async(smem_u32(slot + (2 * j + 1) * NT), ur + c);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    const int64_t first = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    fetch(first);
    int it = 0;
    for (int64_t r = first; r < o.M; r += step, ++it) {
        f32x2 y[CH][4];
        float amax = 0.0f;
        copies_wait();
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            if (t + j * TPR < nchunks) {
                gated_chunk<GELU>(slot[2 * j * NT], slot[(2 * j + 1) * NT], y[j]);
                amax = absmax_nan(amax, chunk_amax(y[j]));
            }
        }
        fetch(r + step); /* the slots have been used up: y depends on all they held */
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            amax = absmax_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
        if constexpr (TPR > 32) {
            float *rd = red[it & 1]; /* alternate buffers: one barrier per row */
            if ((threadIdx.x & 31) == 0)
                rd[threadIdx.x >> 5] = amax;
            __syncthreads();
            amax = rd[0];
#pragma unroll
            for (int w = 1; w < NT / 32; ++w)
                amax = absmax_nan(amax, rd[w]);
        }
        const float s = __fdiv_rn(amax, 448.0f);
        const float rcp = __frcp_rn(s);
        const bool exact_row = rw_exact_row(s, rcp);
        if (t == 0)
            static_cast<float *>(o.S)[r] = s;
        uint2 *qrow = reinterpret_cast<uint2 *>(code_row<OUT_FP8RW>(o, (int)r));
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = t + j * TPR;
            if (c < nchunks)
                qrow[c] = rw_chunk_codes(y[j], s, rcp, exact_row);
        }
    }
}

int device_sms()
{
    static std::atomic<int> sms[64] = {}; /* several host threads may fill an entry, with the same value */
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 148;
    int v = sms[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
            v = 148;
        sms[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

template <int FMT, bool GELU>
static cudaError_t launch_blocks(const GatedArgs &p, const QuantOut &o, cudaStream_t stream)
{
    const int nseg = (o.K / 8 + 31) / 32;
    int wx = 1;
    while (wx < GT / 32 && wx < nseg)
        wx *= 2;
    const int wy = (GT / 32) / wx;
    const int gx = (nseg + wx - 1) / wx;
    int64_t gy = ((int64_t)o.rows + wy - 1) / wy;
    /* Two waves of resident blocks: one wave leaves the SMs that finish first
     * idle (60000 x 1024: 61.6 us against 53.9), four or more restart the loads
     * too often when rows are few (2000 x 4096: 12.0 against 9.9).  Counted by what
     * is resident: NVFP4 with the five blocks of the others, two and a half waves,
     * 32760 x 13824: 454 us against 398, 2047 x 13824: 25.5 against 26.0. */
    int64_t cap = (int64_t)device_sms() * 2 * gated_blocks(FMT) / gx;
    if (cap < 1)
        cap = 1;
    if (gy > cap)
        gy = cap;
    return launch_chained(gated_quantize_kernel<FMT, GELU>, dim3((unsigned)gx, (unsigned)gy), dim3(GT), 0, stream, 1, p,
                          o, wx);
}

template <bool GELU, int NT, int TPR, int CH>
static cudaError_t launch_rows(const GatedArgs &p, const QuantOut &o, cudaStream_t stream)
{
    constexpr int RPB = NT / TPR;
    int64_t blocks = ((int64_t)o.M + RPB - 1) / RPB;
    const int64_t cap = (int64_t)device_sms() * (2048 / NT);
    if (blocks > cap)
        blocks = cap;
    auto kernel = gated_quantize_rowwise_kernel<GELU, NT, TPR, CH>;
    constexpr size_t smem = (size_t)NT * CH * 2 * sizeof(uint4);
    if (smem > 48u * 1024u) {
        static std::atomic<bool> attr_set[64] = {};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess)
            return e;
        if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess)
                return e;
            if (dev >= 0 && dev < 64)
                attr_set[dev].store(true, std::memory_order_release);
        }
    }
    return launch_chained(kernel, dim3((unsigned)blocks), dim3(NT), smem, stream, 1, p, o);
}

template <bool GELU>
static cudaError_t launch_act(int fmt, const GatedArgs &p, const QuantOut &o, cudaStream_t stream)
{
    switch (fmt) {
    case OUT_MXFP8_TC:
        return launch_blocks<OUT_MXFP8_TC, GELU>(p, o, stream);
    case OUT_MXFP8_ROW:
        return launch_blocks<OUT_MXFP8_ROW, GELU>(p, o, stream);
    case OUT_NVFP4:
        return launch_blocks<OUT_NVFP4, GELU>(p, o, stream);
    case OUT_MXFP4:
        return launch_blocks<OUT_MXFP4, GELU>(p, o, stream);
    default:
        break;
    }
    const int nchunks = o.K / 8;
    if (nchunks <= 4 * 32)
        return launch_rows<GELU, 256, 32, 4>(p, o, stream);
    if (nchunks <= 4 * 128)
        return launch_rows<GELU, 128, 128, 4>(p, o, stream);
    if (nchunks <= 4 * 256)
        return launch_rows<GELU, 256, 256, 4>(p, o, stream);
    return launch_rows<GELU, 512, 512, 4>(p, o, stream);
}

cudaError_t launch_gated_quantize(int fmt, bool gelu, const GatedArgs &p, const QuantOut &o, cudaStream_t stream)
{
    if (o.rows == 0)
        return cudaSuccess;
    return gelu ? launch_act<true>(fmt, p, o, stream) : launch_act<false>(fmt, p, o, stream);
}

} // namespace mx
