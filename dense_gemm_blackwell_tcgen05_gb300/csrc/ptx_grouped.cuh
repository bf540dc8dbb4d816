// PTX wrappers that only the grouped kernels need, beside those of ptx.cuh.
#pragma once

#include "ptx.cuh"

namespace gb300 {

// mbar_arrive_cluster without release semantics, for an arrival that hands back
// what this thread has only read: a release at cluster scope first waits for the
// thread's earlier global stores, which such a hand-back does not publish.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}

// Stores `value` at `cluster_addr` and then completes 4 transaction bytes on
// `cluster_bar`, both in one CTA of the cluster (addresses from mapa),
// asynchronously: the completion releases at cluster scope without making
// this thread wait for its SM's outstanding stores, as an arrive.release
// from another CTA does.
__device__ __forceinline__ void st_async_u32(uint32_t cluster_addr, uint32_t value, uint32_t cluster_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(cluster_addr),
               "r"(value), "r"(cluster_bar)
               : "memory");
}

// Four words at once, 16 transaction bytes.
__device__ __forceinline__ void st_async_v4(uint32_t cluster_addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                            uint32_t cluster_bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(cluster_addr),
      "r"(a), "r"(b), "r"(c), "r"(d), "r"(cluster_bar)
      : "memory");
}

// 32 bytes at a 32-byte boundary of global memory, 16 at a 16-byte one.
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
__device__ __forceinline__ void st_global_v4(void* p, const uint32_t* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(x[0], x[1], x[2], x[3]);
}

}  // namespace gb300
