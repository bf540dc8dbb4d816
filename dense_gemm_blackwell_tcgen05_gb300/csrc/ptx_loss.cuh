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

// A warpgroup's registers a thread from here on, within what the block was launched with.
template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 operations in one instruction, each rounded as it would be alone: a += b, and
// x = a x + b with a and b for both.
__device__ __forceinline__ void add_pair(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma_pair(float a, float& x0, float& x1, float b) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, y, x, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(a), "f"(b));
}

// A warp's box of 32 rows of 128 bytes for a store with 128-byte swizzle: pieces `first` ..
// of 16 bytes of this lane's row, N words.
template <uint32_t N>
__device__ __forceinline__ void stage_row(uint32_t box, uint32_t lane, uint32_t first, const uint32_t (&v)[N]) {
#pragma unroll
  for (uint32_t i = 0; i < N / 4; ++i)
    st_shared_v4(box + lane * 128 + (((first + i) ^ (lane & 7u)) << 4), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// The same of 32 rows of 64 bytes with 64-byte swizzle, a whole row.
__device__ __forceinline__ void stage_half_row(uint32_t box, uint32_t lane, const uint32_t (&v)[16]) {
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i)
    st_shared_v4(box + lane * 64 + ((i ^ ((lane >> 1) & 3u)) << 4), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
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
