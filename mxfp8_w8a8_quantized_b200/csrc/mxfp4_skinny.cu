/*
 * mxfp4_skinny.cu -- the MXFP4 linear for few rows (decoding): Y[m, n] =
 * BF16(sum_b 2^(sx[m,b] + sw[n,b]) sum_j x[m,32b+j] w[n,32b+j] + bias[n]) on
 * the sm_100a tensor cores, bound by the weights' way from HBM.
 *
 * With M rows there are 2 M operations per weight, so the floor is the weight:
 * N K (1/2 + 1/32) bytes.  The product is taken transposed: 128 weight rows
 * are the MMA's M dimension and the activation rows (padded to 16, 32, 64 or
 * 128) its N dimension, so no tensor-core work and no shared memory goes to
 * rows that are not there.  The K axis of a 128-row weight tile is split over
 * a cluster of S CTAs where there are fewer tiles than SMs; every CTA stores
 * its FP32 partial rows into the shared memory of the CTA that owns them (row
 * m belongs to CTA m % S), which sums them in the order of the K parts.  No
 * workspace, no atomics: the result does not depend on the order in which
 * CTAs run.  (Laying the received parts over the spent ring, so that two CTAs
 * with 64 or 128 rows share an SM, needs one more cluster barrier and lost on
 * all but the longest K: K = N = 5120, M = 128: 11.0 us against 9.6.)
 *
 * Roles (192 threads): warp 0 TMA producer (a ring of stages, 128 weight rows
 * x 128 bytes = 256 elements each, their scale atoms, and the same K step of
 * the activations), warp 1 scale copies and MMAs (one thread), warps 2..5
 * epilogue.  The kernel is launched chained: while the kernel ahead still
 * runs, it sets up and prefetches its weights into L2.
 *
 * Measured in a captured graph of layers with weights that are not in L2 (us,
 * and the weights' bytes per second as a fraction of the measured copy rate):
 *   K 5120, N 27648   M 1: 15.2 (0.76)   M 64: 16.2   M 128: 18.1
 *   K 5120, N 13824   M 1:  9.7 (0.59)   M 64: 11.3   M 128: 12.6
 *   K 13824, N 5120   M 1:  9.5 (0.61)   M 64: 12.5   M 128: 15.3
 *   K = N = 5120      M 1:  6.1 (0.35)   M 64:  8.4   M 128: 10.4
 *   K = N = 1024      M 1:  2.8          M 64:  4.1   M 128:  4.9 (one K part)
 * (on a GPU where each is 2 to 8 % above the fastest one measured).
 * What is left over the weights' time is the launch, the pipeline's first and
 * last latencies and the cluster's two barriers: about 3 us, as the smallest
 * case shows.
 *
 * Every wait is bounded, as in mxfp8_gemm.cu: on timeout the status word
 * records it, the other roles stop, copies in flight settle, and the kernel
 * returns through its cluster barriers.
 */
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "fused_quant.cuh"
#include "ptx.cuh"
#include "tmap_host.cuh"

namespace mx {

constexpr int SK_THREADS = 192;
constexpr uint32_t SK_SUSPEND_NS = 1000000;
constexpr uint64_t SK_SETTLE_NS = 200000;

__device__ unsigned int g_sk_status = 0; /* bit 0: a bounded wait gave up */

constexpr int SK_MAX_STAGES = 6;
constexpr int SK_MAX_S = 8;

template <int MT>
struct SkCfg {
    static constexpr uint32_t OFF_X = 128 * 128;             /* after 128 weight rows x 256 codes */
    static constexpr uint32_t OFF_SFW = OFF_X + MT * 128;    /* scale atoms: 128 rows x 8 blocks */
    static constexpr uint32_t OFF_SFX = OFF_SFW + 1024;
    static constexpr uint32_t STAGE = OFF_SFX + 1024;
    static constexpr uint32_t SF_COL = MT < 32 ? 32 : MT;
    static constexpr uint32_t SF_STEP = 16;                  /* scale columns per stage */
    static constexpr uint32_t TMEM_COLS = 256;               /* two CTAs per SM fit */
    static_assert(SF_COL + SF_STEP * SK_MAX_STAGES <= TMEM_COLS, "TMEM budget");
    static_assert(STAGE % 1024 == 0, "swizzle atoms");
    /* barriers, then S parts of ceil(MT / S) rows */
    static constexpr uint32_t BAR_BYTES = 256;
    static_assert((2 * SK_MAX_STAGES + 2) * 8 + 8 <= BAR_BYTES, "barriers");
    static constexpr uint32_t fixed_bytes(int S) { return 1024u + BAR_BYTES + (S > 1 ? (MT + SK_MAX_S) * 512u : 0u); }
    /* stages that fit `bytes` of shared memory */
    static constexpr int stages_in(uint32_t bytes, int S)
    {
        return fixed_bytes(S) > bytes ? 0
               : (bytes - fixed_bytes(S)) / STAGE > SK_MAX_STAGES ? SK_MAX_STAGES
                                                                  : (int)((bytes - fixed_bytes(S)) / STAGE);
    }
};
constexpr uint32_t SK_SMEM_ONE = 232448, SK_SMEM_TWO = 115712; /* per CTA, one or two of them per SM */

/*
 * Two CTAs per SM hold all 512 TMEM columns between them and the large GEMM's
 * CTA holds them alone, so the allocation never waits for another CTA as long
 * as shared memory keeps a third one, or one beside the large GEMM (at least
 * 150 KB), off the SM.  It must not wait: CTAs of two clusters could then wait
 * for one another's columns.
 */
template <int MT>
constexpr bool sk_two_per_sm()
{
    using C = SkCfg<MT>;
    for (int S = 1; S <= SK_MAX_S; ++S) {
        const int few = C::stages_in(SK_SMEM_TWO, S), many = C::stages_in(SK_SMEM_ONE, S);
        const uint32_t least = C::fixed_bytes(S) + (uint32_t)(few >= 3 ? few : many) * C::STAGE;
        if (3u * least <= 233472u || least + 153600u <= 233472u) /* 228 KB per SM */
            return false;
    }
    return true;
}
static_assert(sk_two_per_sm<16>() && sk_two_per_sm<32>() && sk_two_per_sm<64>() && sk_two_per_sm<128>(),
              "a third CTA would wait for TMEM");

struct SkParams {
    const __half *bias;
    __nv_bfloat16 *Y;
    int M, N;
    int KB;     /* K steps of 256 */
    int S;      /* CTAs per weight tile */
    int stages; /* of the ring */
    unsigned long long timeout_ns;
};

/* Position in the ring: stage and the parity of its use. */
struct SkRing {
    uint32_t s = 0, use = 0;
    __device__ __forceinline__ void next(int stages)
    {
        if (++s == (uint32_t)stages) {
            s = 0;
            use ^= 1u;
        }
    }
};

__device__ __forceinline__ bool sk_wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns,
                                        volatile uint32_t *abort_flag)
{
    if (mbar_try_wait(bar, parity, SK_SUSPEND_NS))
        return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity, SK_SUSPEND_NS))
            return true;
        if (*abort_flag)
            return false;
        if (globaltimer_ns() - t0 > limit_ns) {
            *abort_flag = 1u;
            atomicOr(&g_sk_status, 1u);
            return false;
        }
    }
}

template <int MT>
__global__ void __launch_bounds__(SK_THREADS) mxfp4_skinny_kernel(const __grid_constant__ CUtensorMap tmap_w,
                                                                  const __grid_constant__ CUtensorMap tmap_x,
                                                                  const __grid_constant__ CUtensorMap tmap_sfw,
                                                                  const __grid_constant__ CUtensorMap tmap_sfx,
                                                                  const SkParams p)
{
    using C = SkCfg<MT>;
    extern __shared__ uint8_t sk_smem[];
    const uint32_t raw = smem_u32(sk_smem);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = sk_smem + (sbase - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const int tile = (int)blockIdx.x / p.S;
    const int m0 = (int)blockIdx.y * MT;
    const int kb0 = p.KB * rank / p.S;
    const int nkb = p.KB * (rank + 1) / p.S - kb0;

    const uint32_t off_bar = (uint32_t)p.stages * C::STAGE, off_part = off_bar + C::BAR_BYTES;
    const uint32_t bar_full = sbase + off_bar;
    const uint32_t bar_empty = bar_full + 8 * SK_MAX_STAGES;
    const uint32_t bar_tfull = bar_empty + 8 * SK_MAX_STAGES;
    const uint32_t bar_drain = bar_tfull + 8;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(smem + off_bar + 8 * (2 * SK_MAX_STAGES + 2));
    volatile uint32_t *abort_flag = tmem_ptr + 1;
    const unsigned long long lim = p.timeout_ns;

    /* K step kb0 + i into stage s */
    auto load = [&](int i, uint32_t s) {
        const uint32_t bar = bar_full + 8 * s, at = sbase + s * C::STAGE;
        mbar_arrive_expect_tx(bar, C::STAGE);
        tma_load_2d(at, &tmap_w, (kb0 + i) * 128, tile * 128, bar);
        tma_load_3d(at + C::OFF_SFW, &tmap_sfw, 0, 2 * (kb0 + i), tile, bar);
        tma_load_2d(at + C::OFF_X, &tmap_x, (kb0 + i) * 128, m0, bar);
        tma_load_3d(at + C::OFF_SFX, &tmap_sfx, 0, 2 * (kb0 + i), m0 / 128, bar);
    };

    if (p.S > 1)
        cluster_arrive(); /* waited for before the first push: every CTA has started */
    if (threadIdx.x == 0) {
        *abort_flag = 0u;
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        mbar_init(bar_tfull, 1);
        mbar_init(bar_drain, 1);
        fence_mbar_init();
        const int pre = min(p.stages, nkb);
        for (int i = 0; i < pre; ++i) {
            tma_prefetch_2d(&tmap_w, (kb0 + i) * 128, tile * 128);
            tma_prefetch_3d(&tmap_sfw, 0, 2 * (kb0 + i), tile);
        }
        grid_wait_ahead();
        for (int i = 0; i < pre; ++i)
            load(i, (uint32_t)i);
    }
    if (warp == 1) {
        /* Ahead of the launch, so that what starts behind this kernel takes none of
         * its TMEM, and ahead of the wait for the kernel before: an SM starts no
         * second CTA while one there may still allocate, and those that started
         * only when the one ahead had ended cost a token 3 us (K = 5120, N = 13824,
         * M = 1: 13.4 us against 10.3 for the linear). */
        tmem_alloc(smem_u32(tmem_ptr), C::TMEM_COLS);
        tmem_relinquish();
        grid_launch_dependents();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_ptr;

    if (warp == 0) {
        if (lane == 0) {
            SkRing at; /* step i refills the stage of step i - stages */
            for (int i = p.stages; i < nkb; ++i, at.next(p.stages)) {
                if (!sk_wait(bar_empty + 8 * at.s, at.use, lim, abort_flag))
                    break;
                load(i, at.s);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_mxf4(128, MT);
            bool ok = true;
            SkRing at;
            for (int i = 0; i < nkb; ++i, at.next(p.stages)) {
                const uint32_t s = at.s, stage = sbase + s * C::STAGE;
                if (!sk_wait(bar_full + 8 * s, at.use, lim, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tsfw = tmem + C::SF_COL + C::SF_STEP * s, tsfx = tsfw + 8;
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    tc_cp_32x128b_warpx4(tsfw + 4u * a, desc_sf_32x16(stage + C::OFF_SFW + 512u * a));
                    tc_cp_32x128b_warpx4(tsfx + 4u * a, desc_sf_32x16(stage + C::OFF_SFX + 512u * a));
                }
                const uint64_t wdesc = desc_kmajor_sw128(stage);
                const uint64_t xdesc = desc_kmajor_sw128(stage + C::OFF_X);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc_mma_mxf4(tmem, wdesc + (uint64_t)(2 * k), xdesc + (uint64_t)(2 * k),
                                idesc_with_sf_id(idesc, 2u * (k & 1)), tsfw + 4u * (k >> 1), tsfx + 4u * (k >> 1),
                                (i | k) != 0);
                tc_commit(bar_empty + 8 * s);
            }
            if (ok) {
                tc_commit(bar_tfull);
            } else {
                /* this thread's MMAs and copies end before TMEM is freed */
                volatile uint32_t own = 0u;
                tc_commit(bar_drain);
                (void)sk_wait(bar_drain, 0u, lim, &own);
            }
        }
    }
    /* ------------------------------------------------ epilogue (warps 2..5) */
    const int q = warp & 3; /* TMEM sub-partition this warp may read */
    const int n = 32 * q + lane;
    const int col = tile * 128 + n;
    float b = 0.0f;
    bool got = false;
    if (warp >= 2) {
        grid_wait_ahead(); /* these threads read the bias and write Y */
        if (p.bias && col < p.N)
            b = __half2float(p.bias[col]);
        got = __all_sync(0xFFFFFFFFu, sk_wait(bar_tfull, 0u, lim, abort_flag));
        tc_fence_after();
    }
    __syncwarp();
    if (p.S > 1)
        cluster_wait();
    const int rows = min(MT, p.M - m0);
    const int own = (rows + p.S - 1) / p.S; /* row slots per part */
    if (got) {
        /* rolled loops: this code runs once per CTA, so its length is paid in
         * instruction fetches (unrolled over MT, 65 cycles per row) */
        __nv_bfloat16 *y = p.Y + (int64_t)m0 * p.N + col;
        const uint32_t part = sbase + off_part + (uint32_t)(rank * own * 128 + n) * 4u;
        int to = 0, slot = 0; /* row m -> CTA m % S, slot m / S of this part */
#pragma unroll 1
        for (int c = 0; c < rows; c += 8) {
            uint32_t acc[8];
            tmem_ld_32x32b_x8_sync(tmem + ((uint32_t)(32 * q) << 16) + c, acc);
            if (p.S == 1) {
#pragma unroll
                for (int j = 0; j < 8; ++j, y += p.N)
                    if (c + j < rows && col < p.N)
                        *y = __float2bfloat16_rn(__uint_as_float(acc[j]) + b);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (c + j < rows)
                        st_cluster_f32(mapa_shared(part + (uint32_t)slot * 512u, (uint32_t)to), __uint_as_float(acc[j]));
                    if (++to == p.S) {
                        to = 0;
                        ++slot;
                    }
                }
            }
        }
        tc_fence_before();
    }
    if (p.S > 1) {
        __syncwarp();
        cluster_sync_all(); /* every part has arrived; nothing remote is touched after this */
        if (warp >= 2 && !*abort_flag) {
            const float *part = reinterpret_cast<const float *>(smem + off_part) + n;
            const int mine = (rows - rank + p.S - 1) / p.S; /* rows of this CTA (<= own) */
            __nv_bfloat16 *y = p.Y + (int64_t)(m0 + rank) * p.N + col;
            const int64_t step = (int64_t)p.S * p.N;
#pragma unroll 1
            for (int i = 0; i < mine; i += 4) {
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                for (int c = 0; c < p.S; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[j] += part[(c * own + min(i + j, mine - 1)) * 128];
#pragma unroll
                for (int j = 0; j < 4; ++j, y += step)
                    if (i + j < mine && col < p.N)
                        *y = __float2bfloat16_rn(s[j] + b);
            }
        }
    }

    __syncthreads();
    if (*abort_flag) {
        /* copies this CTA issued may still be landing in its shared memory */
        if (threadIdx.x == 0) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < SK_SETTLE_NS)
                __nanosleep(1000);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

/* Self-test of sk_wait: a wait on an mbarrier that nothing arrives at gives
 * up after limit_ns and records it as a stalled pipeline would. */
__global__ void sk_wait_selftest_kernel(unsigned long long limit_ns)
{
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0u;
        mbar_init(smem_u32(&bar), 1);
        fence_mbar_init();
        (void)sk_wait(smem_u32(&bar), 0u, limit_ns, &abort_flag);
    }
}

/* ------------------------------------------------------------ host side */
/* Scale atoms [row blocks][kg][512 B]; box = two K groups of one row block. */
static bool sk_scale_map(CUtensorMap *m, const void *base, int64_t rows, int64_t kg)
{
    const cuuint64_t dims[3] = {128, (cuuint64_t)kg, (cuuint64_t)((rows + 127) / 128)};
    const cuuint64_t strides[2] = {512, (cuuint64_t)(kg * 512)};
    const cuuint32_t box[3] = {128, 2, 1};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

/*
 * K parts and ring depth for `tiles` (weight tiles x row tiles).
 *
 * As many parts as leave all CTAs resident at once, since a second wave costs
 * more than a part saves (M = 1, K = 13824, N = 5120: 3 / 6 / 7 parts 10.4 /
 * 9.6 / 13.1 us).  How many clusters of S fit at one CTA per SM is asked of the
 * driver (a cluster stays within one group of SMs, so SMs are left over); twice
 * as many fit where two CTAs share an SM.  No parts where the K steps that they
 * save (0.37 us each) cost less than handing the partial rows over (0.3 us and 16
 * ns per row: K = N = 1024, one or four parts, M = 16: 3.6 / 3.0 us, M = 128: 4.8 /
 * 6.0 us).
 *
 * Up to 32 rows the ring is as deep as two CTAs per SM allow: a CTA of the next
 * launch can then start under the tail of this one (K = N = 5120, M = 1: 5.7 us
 * against 6.4 with the ring of a whole SM).  From 33 rows on a stage is larger
 * and the whole SM's memory is used (K = 5120, N = 13824, M = 128: 11.4 us
 * against 14.1 with three stages), unless there are more CTAs than SMs (N =
 * 27648: 17.2 against 24.3).
 */
template <int MT>
struct SkPlan {
    /* Resident clusters of S CTAs (0: none, S is not used).  Host threads may fill
     * the plan at the same time, with the same values; `ready` publishes them. */
    std::atomic<int> clusters[SK_MAX_S + 1] = {};
    std::atomic<bool> ready{false};

    static constexpr bool SMALL = MT <= 32;
    static bool two(int S) { return SkCfg<MT>::stages_in(SK_SMEM_TWO, S) >= 3; }
    static uint32_t smem(int S, int stages) { return SkCfg<MT>::fixed_bytes(S) + (uint32_t)stages * SkCfg<MT>::STAGE; }

    cudaError_t init(int sms)
    {
        cudaError_t e = cudaFuncSetAttribute(mxfp4_skinny_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)SK_SMEM_ONE);
        for (int S = SK_MAX_S; e == cudaSuccess && S >= 1; --S) {
            int n = sms;
            if (S > 1) {
                cudaLaunchConfig_t cfg = {};
                cudaLaunchAttribute attr[1];
                cfg.gridDim = dim3((unsigned)(S * sms));
                cfg.blockDim = dim3(SK_THREADS);
                cfg.dynamicSmemBytes = smem(S, SkCfg<MT>::stages_in(SK_SMEM_ONE, S));
                attr[0].id = cudaLaunchAttributeClusterDimension;
                attr[0].val.clusterDim.x = (unsigned)S;
                attr[0].val.clusterDim.y = 1;
                attr[0].val.clusterDim.z = 1;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                e = cudaOccupancyMaxActiveClusters(&n, mxfp4_skinny_kernel<MT>, &cfg);
            }
            clusters[S].store(n * (two(S) ? 2 : 1), std::memory_order_relaxed);
        }
        if (e == cudaSuccess)
            ready.store(true, std::memory_order_release);
        return e;
    }
};

template <int MT>
static cudaError_t sk_launch(const CUtensorMap &mw, const CUtensorMap &mx_, const CUtensorMap &msw,
                             const CUtensorMap &msx, SkParams p, int tiles, int mtiles, cudaStream_t stream)
{
    static SkPlan<MT> plans[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    SkPlan<MT> &plan = plans[dev];
    const int sms = device_sms();
    if (!plan.ready.load(std::memory_order_acquire)) {
        e = plan.init(sms);
        if (e != cudaSuccess)
            return e;
    }
    const int64_t work = (int64_t)tiles * mtiles;
    int S = SK_MAX_S < p.KB ? SK_MAX_S : p.KB;
    while (S > 1 && work > plan.clusters[S].load(std::memory_order_relaxed))
        --S;
    const int saved = p.KB - (p.KB + S - 1) / S, rows = p.M < MT ? p.M : MT;
    if (370 * saved < 300 + 16 * rows)
        S = 1;
    p.S = S;
    const bool two = SkPlan<MT>::two(S) && (SkPlan<MT>::SMALL || work * S > sms);
    p.stages = SkCfg<MT>::stages_in(two ? SK_SMEM_TWO : SK_SMEM_ONE, S);
    return launch_chained(mxfp4_skinny_kernel<MT>, dim3((unsigned)(tiles * S), (unsigned)mtiles), dim3(SK_THREADS),
                          SkPlan<MT>::smem(S, p.stages), stream, S, mw, mx_, msw, msx, p);
}

/* Operands as launch_gemm's MXFP4 mode.  Returns 0 ok, 1 tensor-map failure,
 * 2 CUDA error (in *err). */
int launch_mxfp4_skinny(const void *Xq, const void *Xs, int64_t M, int64_t K, const void *Wq, const void *Ws,
                        int64_t N, const void *bias, void *Y, cudaStream_t stream, unsigned long long timeout_ns,
                        cudaError_t *err)
{
    *err = cudaSuccess;
    const int mt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    const int64_t kg = (K + 127) / 128;
    CUtensorMap mw, mxm, msw, msx;
    if (!encode_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, Wq, K / 2, N, K / 2, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&mxm, CU_TENSOR_MAP_DATA_TYPE_UINT8, Xq, K / 2, M, K / 2, 128, (uint32_t)mt,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !sk_scale_map(&msw, Ws, N, kg) || !sk_scale_map(&msx, Xs, M, kg))
        return 1;
    SkParams p;
    p.bias = static_cast<const __half *>(bias);
    p.Y = static_cast<__nv_bfloat16 *>(Y);
    p.M = (int)M;
    p.N = (int)N;
    p.KB = (int)((K + 255) / 256);
    p.S = p.stages = 0; /* sk_launch */
    p.timeout_ns = timeout_ns;
    const int tiles = (int)((N + 127) / 128), mtiles = (int)((M + mt - 1) / mt);
    cudaError_t e = mt == 16   ? sk_launch<16>(mw, mxm, msw, msx, p, tiles, mtiles, stream)
                    : mt == 32 ? sk_launch<32>(mw, mxm, msw, msx, p, tiles, mtiles, stream)
                    : mt == 64 ? sk_launch<64>(mw, mxm, msw, msx, p, tiles, mtiles, stream)
                               : sk_launch<128>(mw, mxm, msw, msx, p, tiles, mtiles, stream);
    if (e != cudaSuccess) {
        *err = e;
        return 2;
    }
    return 0;
}

cudaError_t launch_skinny_wait_selftest(unsigned long long limit_ns, cudaStream_t stream)
{
    sk_wait_selftest_kernel<<<1, 32, 0, stream>>>(limit_ns);
    return cudaGetLastError();
}

/* Reads and clears this file's status word (synchronous). */
cudaError_t read_and_clear_skinny_status(unsigned int *out)
{
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_sk_status, sizeof(unsigned int));
    if (e != cudaSuccess)
        return e;
    return cudaMemcpyToSymbol(g_sk_status, &zero, sizeof(unsigned int));
}

} // namespace mx
