// The losses' products with a piece of the logits' gradient (loss_products.cuh): tiles,
// parts of the reduction, launches.
#include "launch_loss.cuh"
#include "loss_products.cuh"

namespace gb300 {
namespace {

// Columns of a tile: the width in equal tiles of at most `most`, in steps of 32.
uint32_t tile_columns(uint64_t K, uint64_t most) {
  return static_cast<uint32_t>(ceil_div_u64(ceil_div_u64(K, ceil_div_u64(K, most)), 32) * 32);
}

template <int CG, LossOp OP, class T>
int launch(const LossProduct& p, uint32_t nt, uint32_t split, const LaunchCtx& ctx, cudaStream_t stream) {
  using C = LossProductCfg<CG, OP>;
  uint64_t room = 0;
  if (const int rc = loss_room<C, loss_product_kernel<CG, OP, T>, CG>(ctx, &room); rc != GEMM_OK) return rc;
  CUtensorMap g, x;
  if (!operand_map(&g, p.g, p.n, p.M, 1, p.ldg, 0, C::ROWS ? 128 : 64) ||
      !operand_map(&x, p.X, p.K, C::ROWS ? p.n : p.M, 1, p.ldx, 0, 64))
    return GEMM_ERR_LAUNCH;
  const uint64_t tiles = ceil_div_u64(C::ROWS ? p.M : p.n, C::LT) * ceil_div_u64(p.K, nt) * split;
  if (tiles > 0x7FFFFFFFull) return GEMM_ERR_INVALID_ARG;
  LossProductArgs a = {};
  a.M = p.M;
  a.n = p.n;
  a.K = p.K;
  a.count = p.count;
  a.nt = nt;
  a.split = split;
  a.add = p.add ? 1u : 0u;
  a.out = p.out;
  a.ldo = p.ldo;
  a.stride_o = p.stride_o;
  a.status = ctx.status;
  a.timeout_ns = ctx.timeout_ns;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((tiles < room ? tiles : room) * CG));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  loss_attributes(cfg, attr, CG, true);
  note_schedule(cfg.gridDim.x / CG, CG, static_cast<uint32_t>(tiles), 0u, 0u, 0u, 0u);
  if (const cudaError_t e = cudaLaunchKernelEx(&cfg, loss_product_kernel<CG, OP, T>, g, x, a); e != cudaSuccess) {
    note_cuda_error(e);
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

}  // namespace

// Rounds of items, each as long as its stages and a store, and the parts' sums, which are
// written and read again: at most kMostSums of them beyond the first part.
LossRowsPlan loss_rows_plan(uint64_t M, uint64_t n, uint64_t K) {
  constexpr uint64_t kMostSums = 256ull << 20;
  const uint64_t kt = ceil_div_u64(n, 64);
  LossRowsPlan best = {2, 256, 1};
  double least = 1e300;
  for (uint32_t cg = M <= 128 ? 1 : 2; cg >= 1; --cg) {
    const uint32_t nt = tile_columns(K, 128 * cg);
    const uint64_t tiles = ceil_div_u64(M, 128 * cg) * ceil_div_u64(K, nt);
    for (uint64_t split = 1; split <= 152 && split <= ceil_div_u64(kt, 4); ++split) {
      if (split > 1 && split * M * K * 4 > kMostSums) break;
      const uint64_t rounds = ceil_div_u64(tiles * split, kLossSms / cg);
      const double t = static_cast<double>(rounds) * (static_cast<double>(ceil_div_u64(kt, split)) * (cg == 2 ? 0.30 : 0.27) + 1.5) +
                       (cg == 2 ? 2.0 : 0.0) + static_cast<double>(split * M * K) * 8.0 / 5e6;
      if (t < least) {
        least = t;
        best = {cg, nt, static_cast<uint32_t>(split)};
      }
    }
  }
  return best;
}

int launch_loss_rows(const LossProduct& p, const LossRowsPlan& plan, const LaunchCtx& ctx, cudaStream_t stream) {
  return plan.cg == 2 ? launch<2, LossOp::Rows, uint32_t>(p, plan.nt, plan.split, ctx, stream)
                      : launch<1, LossOp::Rows, uint32_t>(p, plan.nt, plan.split, ctx, stream);
}

bool loss_matrix_ok(const void* out, uint64_t ldo, bool out_f32) {
  return ((reinterpret_cast<uintptr_t>(out) | ldo * (out_f32 ? 4 : 2)) & 31u) == 0;
}

int launch_loss_matrix(const LossProduct& p, const LaunchCtx& ctx, cudaStream_t stream) {
  // rounds of tiles, each as long as its loads or its store
  const uint64_t kt = ceil_div_u64(p.M, 64);
  const auto time = [&](uint64_t cg, double stage, double store) {
    const uint64_t tiles = ceil_div_u64(p.n, 128 * cg) * ceil_div_u64(p.K, 128 * cg);
    const double load = static_cast<double>(kt) * stage;
    return static_cast<double>(ceil_div_u64(tiles, kLossSms / cg)) * (load > store ? load : store);
  };
  const bool pair = time(2, 0.30, p.out_f32 ? 2.8 : 1.6) + 2.5 < time(1, 0.27, p.out_f32 ? 1.4 : 1.2);
  const uint32_t nt = tile_columns(p.K, pair ? 256 : 128);
  if (p.out_f32)
    return pair ? launch<2, LossOp::Matrix, uint32_t>(p, nt, 1, ctx, stream)
                : launch<1, LossOp::Matrix, uint32_t>(p, nt, 1, ctx, stream);
  return pair ? launch<2, LossOp::Matrix, uint16_t>(p, nt, 1, ctx, stream)
              : launch<1, LossOp::Matrix, uint16_t>(p, nt, 1, ctx, stream);
}

}  // namespace gb300
