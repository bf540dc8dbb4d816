// Host-side interface of the losses over a vocabulary (not part of the public ABI).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "gemm_host.h"

namespace gb300 {

// Rows A [M, K] and the vocabulary's matrix B [N, K], bf16, and each row's entries: its
// target (top = 0) or a teacher's list of `top`.
struct LossProblem {
  uint32_t M, N, K, top;
  const void* A;
  const void* B;
  uint64_t lda, ldb;
  float scale;                 // of the logits: 1 / temperature for a list
  // a target per row
  const void* targets;         // [M]
  bool target64;
  float smoothing, z_coef;
  // a teacher's list per row
  const void* teacher;         // [M, top] fp32 or bf16
  bool teacher_f32;
  const void* ids;             // [M, top]
  bool ids64;
  uint64_t ld_teacher, ld_ids;
  // forward
  float* loss;                 // [M]
  float* lse_out;              // [M]
  // backward
  const float* dloss;          // [M] at inc_dloss elements
  uint64_t inc_dloss;
  const float* lse;            // [M]
  void* dA;                    // [M, K] (nullptr: not wanted)
  void* dB;                    // [N, K] (nullptr: not wanted)
  uint64_t ld_da, ld_db;
  bool da_f32, db_f32, accumulate;
  void* workspace;
  uint32_t stall_iter;
};

constexpr uint64_t kNoWorkspace = ~0ull;   // for sizes that no memory holds
uint64_t loss_forward_bytes(uint64_t M, uint64_t N, uint64_t K, uint64_t top);
uint64_t loss_backward_bytes(uint64_t M, uint64_t N, uint64_t K, uint64_t top);
int launch_loss_forward(const LossProblem& p, const LaunchCtx& ctx, cudaStream_t stream);
int launch_loss_backward(const LossProblem& p, const LaunchCtx& ctx, cudaStream_t stream);

// The products (loss_kernels.cuh): rows from A or, where fewer than M count, from
// `compact`; B's rows from `B` on.
struct LossArgs;
struct LossOperands {
  const void* A;
  uint64_t lda;
  const void* compact;
  uint64_t ld_compact;
  const void* B;
  uint64_t ldb;
  bool chained;                // the launch follows another kernel of its call
  uint64_t out_rows;           // backward: of the piece of the gradient
};
// A GB300's SMs, not the current device's: a workspace is sized without a device.
constexpr uint64_t kLossSms = 152;
// Which tiles of the logits.
struct LossTiles {
  uint32_t cg, nt;             // CTAs that share a tile of 128 rows each, its columns
  // Partial results a forward product leaves for each row: one for each tile of columns,
  // or, over one block of rows, for each cluster.
  uint64_t slots(uint64_t M, uint64_t N) const {
    const uint64_t columns = (N + nt - 1) / nt;
    return M <= 128 * cg && columns > kLossSms / cg ? kLossSms / cg : columns;
  }
};
// Rounds of tiles over the SMs, each as long as its stages' loads, at 64 bytes a clock into
// an SM, or their MMAs, and about 1000 clocks of a tile's first loads and last results; and
// the launch of pairs.  The width is what fills the last round: 129 rows against 32768 tokens are
// 128 tiles of 256 columns, two rounds of 76 pairs, but 147 of 224.
inline LossTiles loss_tiles(uint64_t M, uint64_t N, uint64_t K) {
  LossTiles best = {1, 128};
  uint64_t least = ~0ull;
  for (uint32_t cg = 1; cg <= 2; ++cg) {
    if (cg == 2 && M <= 128) break;
    const uint64_t rows = M < 128 ? (M + 31) / 32 * 32 : 128;
    for (uint32_t nt = 128 * cg; nt >= 32; nt -= 32) {
      const uint64_t tiles = (M + 128 * cg - 1) / (128 * cg) * ((N + nt - 1) / nt), clusters = kLossSms / cg;
      const uint64_t load = 2 * rows + 2 * nt / cg, mma = 2 * nt;
      const uint64_t t = (tiles + clusters - 1) / clusters * ((K + 63) / 64 * (load > mma ? load : mma) + 1000) +
                         (cg == 2 ? 3800 : 0);
      if (t < least) {
        least = t;
        best = {cg, nt};
      }
    }
  }
  return best;
}
int launch_loss_logits_forward(const LossOperands& o, LossArgs a, const LaunchCtx& ctx, uint32_t* slots,
                               cudaStream_t stream);
int launch_loss_logits_backward(const LossOperands& o, const LossArgs& a, const LaunchCtx& ctx, cudaStream_t stream);

// The products with a piece of the logits' gradient (loss_products.cuh).
struct LossDeal;
struct LossProduct {
  uint32_t M, n, K, width;     // rows at most, the piece's columns, the width, the first piece's columns
  const LossDeal* deal;        // of the items, found by an earlier kernel (nullptr: no row is left out)
  const void *g, *B;           // [M, n], B's rows of the piece
  const void *A, *compact;     // all rows of A, for where none is left out, and those that count
  uint64_t ldg, ldb, lda, ld_compact;
  float* sums;                 // (nullptr: not wanted) [most][M][K]
  uint64_t ld_sums, stride_sums;
  uint32_t most;
  bool add_sums;
  float* sums_db;              // (nullptr: the rows are not to be dealt in parts) [most_db][n][K], rows of ld_sums
  uint64_t stride_db;
  uint32_t most_db;
  void* dA;                    // (nullptr: not wanted) instead of sums where they need no joining
  uint64_t ld_da;
  bool da_f32;
  void* dB;                    // (nullptr: not wanted) [n, K]
  uint64_t ld_db;
  bool db_f32, add_db;
};
// Parts that the sums' reduction over a piece may be dealt in, at most.
uint32_t loss_most_parts(uint64_t M, uint64_t width, uint64_t K);
// Parts that the product to a matrix of few tiles may deal its rows in, at most.
uint32_t loss_most_parts_db(uint64_t M, uint64_t N, uint64_t K);
// Whether the product to the matrix can be stored at `out`: TMA takes rows that start and
// end on 16 bytes.
bool loss_matrix_ok(const void* out, uint64_t ldo, uint64_t K, bool out_f32, bool add);
// What loss_spread_kernel has to know of these launches: CTAs that share a tile, clusters.
struct LossProductPlan {
  uint32_t cg, nt, clusters;
};
int loss_product_plan(const LossProduct& p, const LaunchCtx& ctx, LossProductPlan* plan);
struct LossProductArgs;
LossProductArgs loss_product_args(const LossProduct& p, const LossProductPlan& plan, const LaunchCtx& ctx);
int launch_loss_products(const LossProduct& p, const LossProductPlan& plan, const LaunchCtx& ctx, cudaStream_t stream);

}  // namespace gb300
