// Writes into the shared memory of a cluster's other blocks by the kernels that exchange counts and
// sums there.
//
// A block may be touched only once it has started, and that the blocks of a cluster run side by
// side does not say that all of them have. So such a kernel arrives at the cluster's barrier first
// thing, works on what is its own, and waits just before its first remote store, by when the
// others have long arrived.
#pragma once

#include <cstdint>

namespace pgg {

// First half of the cluster's barrier: this thread has started. Every thread, once. (Nothing that it
// wrote has to be seen by the others, so it orders nothing: 200 tokens of the few-token form 34.0 ->
// 32.7 us against an arrival that releases.)
__device__ __forceinline__ void cluster_started() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}

// Second half: all blocks of the cluster have started. Every thread, before its first remote store.
__device__ __forceinline__ void cluster_all_started() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// A word or a float into the shared memory of a block of the cluster (address from ptx::mapa).
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

}  // namespace pgg
