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

/* Waits for all of this thread's copies. */
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
}

} // namespace mx
