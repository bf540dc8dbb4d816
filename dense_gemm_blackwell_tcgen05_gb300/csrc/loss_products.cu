// The losses' products with a piece of the logits' gradient (loss_products.cuh): tiles and
// launches.
#include "launch_loss.cuh"
#include "loss_products.cuh"

namespace gb300 {
namespace {

// Columns of a tile: the width in equal tiles of at most `most`, in steps of 64, the columns
// of a box of bf16.
uint32_t tile_columns(uint64_t K, uint64_t most) {
  return static_cast<uint32_t>(ceil_div_u64(ceil_div_u64(K, ceil_div_u64(K, most)), 64) * 64);
}

// Tensor map of outputs [batch][rows][K] stored in boxes of 32 rows of 128 bytes.
bool output_map(CUtensorMap* map, void* base, bool f32, uint64_t K, uint64_t rows, uint64_t batch, uint64_t ld,
                uint64_t stride) {
  const uint64_t size = f32 ? 4 : 2;
  const uint64_t dims[3] = {K, rows, batch};
  const uint64_t strides[2] = {ld * size, (batch > 1 ? stride : ld) * size};
  const uint32_t box[3] = {static_cast<uint32_t>(128 / size), 32, 1};
  return encode_map_3d(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int CG>
int room_of(bool f32, const LaunchCtx& ctx, uint64_t* room) {
  using C = LossProductCfg<CG>;
  return f32 ? loss_room<C, loss_product_kernel<CG, uint32_t>, CG>(ctx, room)
             : loss_room<C, loss_product_kernel<CG, uint16_t>, CG>(ctx, room);
}

template <int CG, class T>
int launch(const LossProduct& p, const LossProductPlan& plan, const LaunchCtx& ctx, cudaStream_t stream) {
  using C = LossProductCfg<CG>;
  uint64_t room = 0;
  if (const int rc = room_of<CG>(p.db_f32, ctx, &room); rc != GEMM_OK) return rc;
  LossMaps m = {};
  if (!operand_map(&m.g_rows, p.g, p.n, p.M, 1, p.ldg, 0, 128) || !operand_map(&m.g_columns, p.g, p.n, p.M, 1, p.ldg, 0, 64) ||
      !operand_map(&m.B, p.B, p.K, p.n, 1, p.ldb, 0, 64) || !operand_map(&m.A, p.A, p.K, p.M, 1, p.lda, 0, 64) ||
      !operand_map(&m.compact, p.compact, p.K, p.M, 1, p.ld_compact, 0, 64) ||
      (p.sums != nullptr && !output_map(&m.sums, p.sums, true, p.K, p.M, p.most, p.ld_sums, p.stride_sums)) ||
      (p.sums_db != nullptr && !output_map(&m.sums_db, p.sums_db, true, p.K, p.n, p.most_db, p.ld_sums, p.stride_db)) ||
      (p.dA != nullptr && !output_map(&m.dA, p.dA, p.da_f32, p.K, p.M, 1, p.ld_da, 0)) ||
      (p.dB != nullptr && !output_map(&m.dB, p.dB, p.db_f32, p.K, p.n, 1, p.ld_db, 0)))
    return GEMM_ERR_LAUNCH;
  const uint64_t columns = ceil_div_u64(p.K, plan.nt);
  const uint64_t tiles = (p.sums != nullptr ? ceil_div_u64(p.M, C::LT) * p.most : 0) * columns +
                         (p.dB != nullptr ? ceil_div_u64(p.n, C::LT) * (p.sums_db != nullptr ? p.most_db : 1) : 0) * columns;
  if (tiles > 0x7FFFFFFFull) return GEMM_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.clusters * CG);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  loss_attributes(cfg, attr, CG, true);
  note_schedule(plan.clusters, CG, static_cast<uint32_t>(tiles), 0u, 0u, 0u, 0u);
  if (const cudaError_t e = cudaLaunchKernelEx(&cfg, loss_product_kernel<CG, T>, m, loss_product_args(p, plan, ctx));
      e != cudaSuccess) {
    note_cuda_error(e);
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

}  // namespace

uint32_t loss_most_parts(uint64_t M, uint64_t width, uint64_t K) {
  constexpr uint64_t kMostSums = 128ull << 20;
  const uint64_t by_size = kMostSums / (4 * M * (K > 0 ? K : 1)), by_length = ceil_div_u64(width, 4 * 64);
  const uint64_t n = by_size < by_length ? by_size : by_length;
  return static_cast<uint32_t>(n < 1 ? 1 : n > 32 ? 32 : n);
}

uint32_t loss_most_parts_db(uint64_t M, uint64_t N, uint64_t K) {
  const uint64_t tiles = ceil_div_u64(N, 128) * ceil_div_u64(K > 0 ? K : 1, 128), by_length = ceil_div_u64(M, 64) / 8;
  const uint64_t n = kLossSms / tiles < by_length ? kLossSms / tiles : by_length;
  return static_cast<uint32_t>(n < 1 ? 1 : n);
}

bool loss_matrix_ok(const void* out, uint64_t ldo, uint64_t K, bool out_f32, bool add) {
  // TMA leaves out what lies past a row's end by pieces of 16 bytes, and adds in the output's
  // type: bf16 would be rounded before it is added
  return ((reinterpret_cast<uintptr_t>(out) | ldo * (out_f32 ? 4 : 2) | K * (out_f32 ? 4 : 2)) & 15u) == 0 &&
         (out_f32 || !add);
}

int loss_product_plan(const LossProduct& p, const LaunchCtx& ctx, LossProductPlan* plan) {
  // rounds of items, each as long as its stages, or a tile's store
  // (pairs halve the loads of the product to the matrix: 64 rows, kept in two halves, 131072 tokens
  // of width 4096: 579 us, 638 on single CTAs)
  const auto time = [&](uint64_t cg, double stage, double store) {
    const uint64_t cb = ceil_div_u64(p.K, 128 * cg);
    double t = 0.0;
    if (p.sums != nullptr)
      t += static_cast<double>(ceil_div_u64(p.M, 128 * cg) * cb * ceil_div_u64(p.width, 64)) * stage;
    if (p.dB != nullptr) {
      const double load = static_cast<double>(ceil_div_u64(p.M, 64)) * stage;
      t += static_cast<double>(ceil_div_u64(p.width, 128 * cg) * cb) * (load > store ? load : store);
    }
    return t * static_cast<double>(cg) / static_cast<double>(kLossSms);
  };
  const bool pair = time(2, 0.30, p.db_f32 ? 2.8 : 1.6) + 2.5 < time(1, 0.27, p.db_f32 ? 1.4 : 1.2);
  plan->cg = pair ? 2 : 1;
  plan->nt = tile_columns(p.K, 128 * plan->cg);
  uint64_t room = 0;
  const int rc = pair ? room_of<2>(p.db_f32, ctx, &room) : room_of<1>(p.db_f32, ctx, &room);
  plan->clusters = static_cast<uint32_t>(room);
  return rc;
}

LossProductArgs loss_product_args(const LossProduct& p, const LossProductPlan& plan, const LaunchCtx& ctx) {
  LossProductArgs a = {};
  a.M = p.M;
  a.n = p.n;
  a.K = p.K;
  a.deal = p.deal;
  a.nt = plan.nt;
  a.width = p.width;
  a.most = p.most;
  a.most_db = p.sums_db != nullptr ? p.most_db : 1u;
  a.rows = p.sums != nullptr ? 1u : 0u;
  a.direct = p.dA == nullptr ? 0u : p.da_f32 ? 2u : 1u;
  a.matrix = p.dB != nullptr ? 1u : 0u;
  a.add_sums = p.add_sums ? 1u : 0u;
  a.add_db = p.add_db ? 1u : 0u;
  a.db_cost = p.db_f32 ? 10u : 6u;
  a.unit = loss_unit(a, 128u * plan.cg);
  a.status = ctx.status;
  a.timeout_ns = ctx.timeout_ns;
  return a;
}

int launch_loss_products(const LossProduct& p, const LossProductPlan& plan, const LaunchCtx& ctx, cudaStream_t stream) {
  if (plan.cg == 2)
    return p.db_f32 ? launch<2, uint32_t>(p, plan, ctx, stream) : launch<2, uint16_t>(p, plan, ctx, stream);
  return p.db_f32 ? launch<1, uint32_t>(p, plan, ctx, stream) : launch<1, uint16_t>(p, plan, ctx, stream);
}

}  // namespace gb300
