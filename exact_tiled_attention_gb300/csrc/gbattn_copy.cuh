// gbattn_copy.cuh -- asynchronous copies of 16 bytes from global into shared
// memory, by groups in the order of their issue (the kernels around a paged
// cache keep rows on their way with them).
#pragma once

#include <stdint.h>

namespace gbattn {

// An asynchronous copy of 16 bytes into shared memory, past L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

}  // namespace gbattn
