// Grouped products that reduce over the grouped rows: the gradient to the
// weights (Op::Sum of grouped_kernels.cuh), and the fill of an empty reduction.
#include "launch_grouped.cuh"

namespace gb300 {
namespace {

template <int CG, uint32_t NT, Op OP, bool OUT32>
int sum_impl(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  using C = GroupedCfg<CG, OP, true, true, NT, OUT32>;
  CUtensorMap tmA, tmD;
  static_assert(p_box_rows<C, true>() == q_box_rows<C, true>(), "either operand in either place");
  if (!operand_map(&tmA, p.A, p.K, p.M, 1, p.lda, 0, p_box_rows<C, true>()) ||
      !operand_map(&tmD, p.dD, p.N, p.M, 1, p.ldd, 0, p_box_rows<C, true>()))
    return GEMM_ERR_LAUNCH;
  GroupedArgs a = {};
  a.L = C::LANE ? p.N : p.K;
  a.C = C::LANE ? p.K : p.N;
  a.K = p.M;
  a.groups = p.groups;
  a.offsets = p.offsets;
  a.out = p.out;
  a.ldo = p.ldo;
  a.stride_o = p.stride_o;
  a.fmt = 1;
  a.status = ctx.status;
  a.timeout_ns = ctx.timeout_ns;
  a.stall_iter = p.stall_iter;
  const uint64_t tiles = ceil_div_u64(a.L, C::LT) * sum_column_tiles<C, NT>(a.C) * p.groups;
  if (tiles > 0x7FFFFFFFull) return GEMM_ERR_INVALID_ARG;
  return launch_grouped<CG, OP, true, true, NT, OUT32>(C::LANE ? tmD : tmA, C::LANE ? tmA : tmD, a, tiles, ctx, stream);
}

// bf16 output rows that start on 16 bytes but not all on 32 (a pitch of 8 columns
// more than a multiple of 16, say): with 32 columns of a row in a warp, half of the
// sectors it stores are partial, and those cost most of the call where the store
// bounds it.  With the rows in the lanes none is but a row's ends.  Measured, us,
// columns / rows in the lanes: 79 groups of 1496 x 3288, 427 rows in all: 253 /
// 154; 24 groups of 1040 x 2056, 171 rows each: 44.5 / 41.3.  Rows of whole sectors
// stay with their columns in the lanes, whose stores touch fewer lines: 24 groups
// of 608 x 3584, 186 rows each: 34 / 43.
bool rows_in_lanes(const GroupedProblem& p) {
  if (p.out_f32 || p.K % 8 != 0) return false;
  const uint64_t starts = reinterpret_cast<uintptr_t>(p.out) | 2 * p.ldo | 2 * p.stride_o;
  return (starts & 15u) == 0 && (starts & 31u) != 0;
}

template <int CG, uint32_t NT>
int sum_pick(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  if (rows_in_lanes(p))
    return p.accumulate ? sum_impl<CG, NT, Op::SumLaneAdd, false>(p, ctx, stream)
                        : sum_impl<CG, NT, Op::SumLane, false>(p, ctx, stream);
  if (p.accumulate)
    return p.out_f32 ? sum_impl<CG, NT, Op::SumAdd, true>(p, ctx, stream)
                     : sum_impl<CG, NT, Op::SumAdd, false>(p, ctx, stream);
  return p.out_f32 ? sum_impl<CG, NT, Op::Sum, true>(p, ctx, stream)
                   : sum_impl<CG, NT, Op::Sum, false>(p, ctx, stream);
}

template <class T>
__global__ void grouped_zero_kernel(T* out, const int32_t* offsets, uint32_t groups, uint32_t rows,
                                    uint32_t cols, uint64_t ldo, uint64_t stride_o) {
  uint64_t lo = 0, hi = static_cast<uint64_t>(rows) * (offsets != nullptr ? 1u : groups);
  if (offsets != nullptr) {
    const int32_t first = min(max(offsets[0], 0), static_cast<int32_t>(rows));
    int32_t last = first;
    for (uint32_t e = 1; e <= groups; ++e) last = max(last, min(offsets[e], static_cast<int32_t>(rows)));
    lo = static_cast<uint64_t>(first);
    hi = static_cast<uint64_t>(last);
  }
  const uint64_t total = (hi - lo) * cols;
  for (uint64_t i = blockIdx.x * static_cast<uint64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<uint64_t>(gridDim.x) * blockDim.x) {
    const uint64_t r = lo + i / cols, c = i % cols;
    out[(r / rows) * stride_o + (r % rows) * ldo + c] = T(0);
  }
}

}  // namespace

int launch_grouped_wgrad(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  // The pair's tiles of 256 x 256 or one CTA's of 128 x 128, by the time of either:
  // rounds of tiles, each as long as its loads (a stage of 64 rows as in the products
  // by rows) or its store, whichever is longer, and 2.5 us for a cluster launch.  Over
  // 110 draws (1 to 16384 rows, 4 to 128 groups, sides of 256 to 4096) the choice is
  // 0.4 % slower in the mean than the better of the two.  Measured, us, one CTA /
  // pair: 24 groups of 1040 x 2056, 171 rows each, bf16 48.5 / 41.3; 84 of 1920 x
  // 2120, 88 rows, bf16 194 / 158; 85 of 488 x 312, 40 rows, bf16 13.3 / 14.1; 8 of
  // 512 x 512, 1024 rows, bf16 8.8 / 12.5; 16 of 1040 x 2056, fp32, 64 rows 29.4 /
  // 33.1, 256 rows 43.2 / 40.5.
  const uint64_t stages = ceil_div_u64(ceil_div_u64(p.M, p.groups), 64);
  const auto time = [&](uint64_t side, uint64_t clusters, double stage, double store) {
    const uint64_t tiles = ceil_div_u64(p.K, side) * ceil_div_u64(p.N, side) * p.groups;
    const double load = static_cast<double>(stages) * stage;
    return static_cast<double>(ceil_div_u64(tiles, clusters)) * (load > store ? load : store);
  };
  const uint64_t sms = static_cast<uint64_t>(ctx.num_sms);
  const bool pair = time(256, sms / 2, 0.30, p.out_f32 ? 2.8 : 1.6) + 2.5 < time(128, sms, 0.27, p.out_f32 ? 1.4 : 1.2);
  return pair ? sum_pick<2, 256>(p, ctx, stream) : sum_pick<1, 128>(p, ctx, stream);
}

int launch_grouped_zero(void* out, bool f32, const int32_t* offsets, uint32_t groups, uint32_t rows,
                        uint32_t cols, uint64_t ldo, uint64_t stride_o, const LaunchCtx& ctx,
                        cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(4 * ctx.num_sms);
  if (f32)
    grouped_zero_kernel<<<grid, 256, 0, stream>>>(static_cast<uint32_t*>(out), offsets, groups, rows, cols,
                                                  ldo, stride_o);
  else
    grouped_zero_kernel<<<grid, 256, 0, stream>>>(static_cast<uint16_t*>(out), offsets, groups, rows, cols,
                                                  ldo, stride_o);
  if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) {
    note_cuda_error(e);
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

}  // namespace gb300
