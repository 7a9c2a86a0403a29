/*
 * async_copy.cuh -- per-thread asynchronous 16-byte copies from global to
 * shared memory (cp.async).  A thread that copies into slots which only it
 * reads needs no barrier: it waits for its own copies.
 */
#pragma once

#include <cstdint>

namespace mx {

__device__ __forceinline__ void copy16_async(uint32_t smem, const void *global)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(global) : "memory");
}

/*
 * Prefetch of the line at `p` into L2.  Allowed ahead of grid_wait_ahead(): it
 * returns no value, and L2 is where all SMs' writes meet, so a later load sees what the
 * kernel ahead has written since.
 */
__device__ __forceinline__ void prefetch_l2(const void *p)
{
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

/* Waits for all of this thread's copies. */
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
}

} // namespace mx
