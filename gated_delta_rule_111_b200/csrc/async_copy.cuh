// Asynchronous copies from global to shared memory by single threads (cp.async):
// each thread waits for its own, in groups, in the order they were issued.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn2 {

__device__ __forceinline__ uint32_t smem_address(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <int BYTES> __device__ __forceinline__ void copy_async(uint32_t smem, const void *global) {
    static_assert(BYTES == 4 || BYTES == 8 || BYTES == 16, "sizes of cp.async");
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(global) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem), "l"(global), "n"(BYTES) : "memory");
}
// The same of which only the first `bytes` are read; the rest of the destination is zero.
template <int BYTES> __device__ __forceinline__ void copy_async_part(uint32_t smem, const void *global, int bytes) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(global), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem), "l"(global), "n"(BYTES), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's newest groups are still in flight.
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void load_shared(uint32_t smem, uint4 &v) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem) : "memory");
}
__device__ __forceinline__ void load_shared(uint32_t smem, uint2 &v) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(smem) : "memory");
}
__device__ __forceinline__ void load_shared(uint32_t smem, unsigned long long &a, unsigned long long &b) {
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(smem) : "memory");
}
__device__ __forceinline__ void store_shared(uint32_t smem, unsigned long long v) {
    asm volatile("st.shared.u64 [%0], %1;" ::"r"(smem), "l"(v) : "memory");
}
template <int BYTES> __device__ __forceinline__ void zero_shared(uint32_t smem) {
#pragma unroll
    for (int i = 0; i < BYTES; i += 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(smem + i), "r"(0) : "memory");
}

}  // namespace gdn2
