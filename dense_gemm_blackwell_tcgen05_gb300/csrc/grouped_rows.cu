// Grouped products whose output rows are the grouped rows: the forward
// product and its gradient to the rows (Op::Rows of grouped_kernels.cuh).
#include "launch_grouped.cuh"

namespace gb300 {
namespace {

// X [M, K'] times each group's matrix; L output columns, K' reduced.
template <bool P_MN, bool OUT32>
int rows_impl(const GroupedProblem& p, const void* X, uint64_t ldx, uint32_t L, uint32_t K,
              const LaunchCtx& ctx, cudaStream_t stream) {
  constexpr int CG = 1;
  constexpr uint32_t NT = 128;
  using C = GroupedCfg<CG, Op::Rows, P_MN, false, NT, OUT32>;
  CUtensorMap tmP, tmQ;
  if (!operand_map(&tmP, p.B, p.K, p.N, p.groups, p.ldb, p.stride_b, p_box_rows<C, P_MN>()) ||
      !operand_map(&tmQ, X, K, p.M, 1, ldx, 0, q_box_rows<C, false>()))
    return GEMM_ERR_LAUNCH;
  GroupedArgs a = {};
  a.L = L;
  a.C = p.M;
  a.K = K;
  a.groups = p.groups;
  a.offsets = p.offsets;
  a.out = p.out;
  a.ldo = p.ldo;
  a.fmt = 1;
  a.status = ctx.status;
  a.timeout_ns = ctx.timeout_ns;
  a.stall_iter = p.stall_iter;
  // at most M / NT full tiles and one ragged one for each group with rows
  const uint64_t touched = p.M < p.groups ? p.M : p.groups;
  const uint64_t tiles = (p.M / NT + touched) * ceil_div_u64(L, C::LT);
  return launch_grouped<CG, Op::Rows, P_MN, false, NT, OUT32>(tmP, tmQ, a, tiles, ctx, stream);
}

}  // namespace

int launch_grouped_forward(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  return p.out_f32 ? rows_impl<false, true>(p, p.A, p.lda, p.N, p.K, ctx, stream)
                   : rows_impl<false, false>(p, p.A, p.lda, p.N, p.K, ctx, stream);
}

int launch_grouped_dgrad(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  return p.out_f32 ? rows_impl<true, true>(p, p.dD, p.ldd, p.K, p.N, ctx, stream)
                   : rows_impl<true, false>(p, p.dD, p.ldd, p.K, p.N, ctx, stream);
}

}  // namespace gb300
