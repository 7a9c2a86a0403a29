/*
 * capi_util.cuh -- what the C-ABI entry points share: limits, alignment
 * checks and the mapping of CUDA errors to statuses.
 */
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "mxfp8.h"

namespace mx {

/* Bound for every pipeline wait inside a kernel. */
constexpr unsigned long long kWaitLimitNs = 4000000000ull;

/* Largest extents the kernels index with 32-bit tile arithmetic. */
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxK = (int64_t)1 << 20;

static inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

static inline size_t round_up(size_t v, size_t a)
{
    return (v + a - 1) / a * a;
}

static inline mxfp8_status from_cuda(cudaError_t e)
{
    return e == cudaSuccess ? MXFP8_OK : MXFP8_ERR_CUDA;
}

} // namespace mx
