// Host-side interface of the grouped products and the Newton-Schulz
// orthogonalisation (not part of the public ABI).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "gemm_host.h"

namespace gb300 {

// The current device's launch context with the watchdog limit for a
// reduction of K set (a gemm_status_t), whether `p` is memory it can address,
// and the calling thread's pending stall request (gemm_debug_stall_next_launch).
int launch_context(int64_t K, LaunchCtx* ctx);
bool device_pointer_ok(const void* p, const LaunchCtx& ctx);
uint32_t take_stall_request();

// encode_map_3d with the swizzle chosen.
bool encode_map_3d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base,
                   const uint64_t (&dims)[3], const uint64_t (&strides)[2], const uint32_t (&box)[3],
                   CUtensorMapSwizzle swizzle);

// Rows of X sorted by group; W [groups, N, K] bf16.
struct GroupedProblem {
  uint32_t M, N, K, groups;          // rows in all, the matrices' rows and columns, groups
  const int32_t* offsets;            // device, [groups + 1]
  const void* A;                     // [M, K] (forward, weight gradient)
  const void* B;                     // [groups, N, K] (forward, row gradient)
  const void* dD;                    // [M, N] (gradients)
  void* out;
  uint64_t lda, ldb, stride_b, ldd;  // pitches of A, B, dD and B's matrix stride, in elements
  uint64_t ldo, stride_o;            // of the output
  bool out_f32, accumulate;
  uint32_t stall_iter;
};

int launch_grouped_forward(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream);
int launch_grouped_dgrad(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream);
int launch_grouped_wgrad(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream);
// Zeros rows offsets[0] .. offsets[groups] - 1 (offsets != nullptr) of an
// [rows, cols] output, or all of a [groups, rows, cols] one: an empty reduction.
int launch_grouped_zero(void* out, bool f32, const int32_t* offsets, uint32_t groups, uint32_t rows,
                        uint32_t cols, uint64_t ldo, uint64_t stride_o, const LaunchCtx& ctx,
                        cudaStream_t stream);

struct NewtonSchulzProblem {
  uint32_t batch, rows, cols;
  const void* G;
  bool g_f32;
  uint64_t ldg, stride_g;
  void* out;
  bool out_f32;
  uint64_t ldo, stride_o;
  int steps;
  float a, b, c, eps;
  void* workspace;
};
uint64_t newton_schulz_bytes(uint64_t batch, uint64_t rows, uint64_t cols);
int launch_newton_schulz(const NewtonSchulzProblem& p, const LaunchCtx& ctx, cudaStream_t stream);

}  // namespace gb300
