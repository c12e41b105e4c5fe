// la_async_copy.cuh — copies to shared memory that the copying thread waits for
// itself (cp.async groups), for rings that no other thread reads.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace la {

// 16 bytes to shared memory, asynchronously; zeros where !ok
__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool ok) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}

}  // namespace la
