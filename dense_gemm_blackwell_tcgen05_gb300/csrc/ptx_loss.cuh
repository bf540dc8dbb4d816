// PTX wrappers that only the losses' kernels need, beside those of ptx.cuh.
#pragma once

#include "gemm_kernels.cuh"
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

// warp_wait for a warp that walks its loop together: every lane probes, and all decide alike,
// so that what follows stays uniform (its addresses in uniform registers, where the tensor
// core's instructions take them).
__device__ __forceinline__ bool uniform_wait(uint32_t bar, uint32_t parity, const Watchdog& wd, uint32_t site, uint32_t lane) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t n = 1;; ++n) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((n & 31u) == 0) {
      if (__any_sync(0xffffffffu, *wd.abort_flag != 0u)) return false;
      if (__any_sync(0xffffffffu, global_timer_ns() - t0 > wd.timeout_ns)) {
        if (lane == 0) {
          *wd.abort_flag = 1u;
          report_error(wd.status, kDevTimeout, site);
        }
        return false;
      }
    }
  }
}

// A ring's stage and the parity of its round.
struct RingStage {
  uint32_t s = 0, round = 0;
  template <uint32_t STAGES>
  __device__ __forceinline__ void next() {
    if (++s == STAGES) s = 0, round ^= 1u;
  }
};

}  // namespace gb300
