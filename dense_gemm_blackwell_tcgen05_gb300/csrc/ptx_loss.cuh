// PTX wrappers that only the losses' kernels need, beside those of ptx.cuh.
#pragma once

#include "ptx.cuh"

namespace gb300 {

// 3-D tiled store from shared memory, and the same added to what the destination holds (in
// the tensor map's type, rounded to nearest), tracked by the bulk async-group of the
// issuing thread.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A warp's box of 32 rows of 128 bytes for a store with 128-byte swizzle: pieces `first` ..
// of 16 bytes of this lane's row, N words.
template <uint32_t N>
__device__ __forceinline__ void stage_row(uint32_t box, uint32_t lane, uint32_t first, const uint32_t (&v)[N]) {
#pragma unroll
  for (uint32_t i = 0; i < N / 4; ++i)
    st_shared_v4(box + lane * 128 + (((first + i) ^ (lane & 7u)) << 4), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

}  // namespace gb300
