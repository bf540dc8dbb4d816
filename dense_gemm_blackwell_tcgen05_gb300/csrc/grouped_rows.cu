// Grouped products whose output rows are the grouped rows: the forward
// product and its gradient to the rows (Op::Rows of grouped_kernels.cuh).
#include "launch_grouped.cuh"

namespace gb300 {
namespace {

// The most tiles a launch can have: M / NT full ones and a ragged one for each
// group that can have rows.
uint64_t most_tiles(const GroupedProblem& p, uint64_t nt, uint64_t lt, uint32_t L) {
  const uint64_t touched = p.M < p.groups ? p.M : p.groups;
  const uint64_t blocks = p.M / nt + touched;
  return (blocks < p.M ? blocks : p.M) * ceil_div_u64(L, lt);
}

// X [M, K'] times each group's matrix; L output columns, K' reduced.
template <int CG, uint32_t NT, bool P_MN, bool OUT32, uint32_t SPLIT = 1>
int rows_impl(const GroupedProblem& p, const void* X, uint64_t ldx, uint32_t L, uint32_t K,
              const LaunchCtx& ctx, cudaStream_t stream) {
  using C = GroupedCfg<CG, Op::Rows, P_MN, false, NT, OUT32, SPLIT>;
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
  const uint64_t tiles = most_tiles(p, NT, C::LT, L);
  return launch_grouped<CG, Op::Rows, P_MN, false, NT, OUT32, SPLIT>(tmP, tmQ, a, tiles, ctx, stream);
}

// Which tiles.  A launch takes its rounds of tiles (those of all groups over
// the CTAs or pairs that run at once), each as long as its loads: a stage of 64 k
// is 24 KB for 64 rows and 128 columns, 32 KB for 128 rows, and 32 KB in each CTA
// of a pair for 256 rows and 256 columns, at 64 bytes a clock from L2 into an SM
// 0.20, 0.27 and 0.27 us.  So wide tiles move least for a product, narrow ones
// leave least of a ragged group empty and spread over most SMs.  0.24, 0.27 and
// 0.30 us and 2 us for a cluster launch fit best: over 365 draws (1 to 16384
// rows, 4 to 128 groups, sides of 256 to 4096) the choice is 0.8 % slower in
// the mean than the best of the three.  Measured, us, 64 rows / 128 / a pair:
// 8 groups of 1024 x 1024, 256 rows each: 11.2 / 11.3 / 11.0, 512: 19.1 / 13.8 /
// 16.0, 1024: 30.1 / 22.4 / 17.9; 32 groups of 4096 x 2048, 4 rows: 80 / 82 / 89,
// 32: 90 / 88 / 93, 256: 215 / 141 / 114; 61 of 399 x 1736, 52 rows: 22.4 / 24.5
// / 24.7.
template <bool P_MN, bool OUT32>
int rows_pick(const GroupedProblem& p, const void* X, uint64_t ldx, uint32_t L, uint32_t K,
              const LaunchCtx& ctx, cudaStream_t stream) {
  const uint64_t touched = p.M < p.groups ? p.M : p.groups;   // groups that can have rows
  // Few tiles and a long reduction: a cluster of CTAs shares it.  A cluster
  // launch and the exchange cost 4.5 us, four CTAs save 0.14 us for each 64 k,
  // two 0.09.  Measured, us, one CTA / two / four, 8 groups, one row in all: 1024
  // x 1024: 6.9 / 9.5 / 9.3, 338 x 2360: 11.3 / 12.2 / 10.6, 256 x 4096: 16.1 /
  // 14.6 / 12.0, 2048 x 4096: 16.8 / 15.4 / 13.4.
  if (K >= 36 * 64) {
    const uint64_t narrow = most_tiles(p, 64, 128, L);
    uint64_t room = 0;
    if (narrow <= static_cast<uint64_t>(ctx.num_sms / 4)) {
      if (const int rc = grouped_room<1, Op::Rows, P_MN, false, 64, OUT32, 4>(ctx, &room); rc != GEMM_OK) return rc;
      if (narrow <= room) return rows_impl<1, 64, P_MN, OUT32, 4>(p, X, ldx, L, K, ctx, stream);
    }
    if (narrow <= static_cast<uint64_t>(ctx.num_sms / 2) && K >= 50 * 64) {
      if (const int rc = grouped_room<1, Op::Rows, P_MN, false, 64, OUT32, 2>(ctx, &room); rc != GEMM_OK) return rc;
      if (narrow <= room) return rows_impl<1, 64, P_MN, OUT32, 2>(p, X, ldx, L, K, ctx, stream);
    }
  }
  const auto time = [&](uint64_t nt, uint64_t lt, uint64_t clusters, double stage) {
    // a group's last tile is half full on average
    const uint64_t blocks = p.M / nt + touched / 2;
    const uint64_t tiles = (blocks > touched ? blocks : touched) * ceil_div_u64(L, lt);
    return static_cast<double>(ceil_div_u64(tiles, clusters) * ceil_div_u64(K, 64)) * stage;
  };
  const uint64_t sms = static_cast<uint64_t>(ctx.num_sms);
  const double narrow = time(64, 128, sms, 0.24), wide = time(128, 128, sms, 0.27),
               pair = time(256, 256, sms / 2, 0.30) + 2.0;
  if (pair < wide && pair < narrow) return rows_impl<2, 256, P_MN, OUT32>(p, X, ldx, L, K, ctx, stream);
  return wide < narrow ? rows_impl<1, 128, P_MN, OUT32>(p, X, ldx, L, K, ctx, stream)
                       : rows_impl<1, 64, P_MN, OUT32>(p, X, ldx, L, K, ctx, stream);
}

}  // namespace

int launch_grouped_forward(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  return p.out_f32 ? rows_pick<false, true>(p, p.A, p.lda, p.N, p.K, ctx, stream)
                   : rows_pick<false, false>(p, p.A, p.lda, p.N, p.K, ctx, stream);
}

int launch_grouped_dgrad(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  return p.out_f32 ? rows_pick<true, true>(p, p.dD, p.ldd, p.K, p.N, ctx, stream)
                   : rows_pick<true, false>(p, p.dD, p.ldd, p.K, p.N, ctx, stream);
}

}  // namespace gb300
