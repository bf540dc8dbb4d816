// Grouped products that reduce over the grouped rows: the gradient to the
// weights (Op::Sum of grouped_kernels.cuh), and the fill of an empty reduction.
#include "launch_grouped.cuh"

namespace gb300 {
namespace {

template <int CG, uint32_t NT, Op OP, bool OUT32>
int sum_impl(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  using C = GroupedCfg<CG, OP, true, true, NT, OUT32>;
  CUtensorMap tmP, tmQ;
  if (!operand_map(&tmP, p.A, p.K, p.M, 1, p.lda, 0, p_box_rows<C, true>()) ||
      !operand_map(&tmQ, p.dD, p.N, p.M, 1, p.ldd, 0, q_box_rows<C, true>()))
    return GEMM_ERR_LAUNCH;
  GroupedArgs a = {};
  a.L = p.K;
  a.C = p.N;
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
  const uint64_t tiles = ceil_div_u64(p.K, C::LT) * ceil_div_u64(p.N, NT) * p.groups;
  if (tiles > 0x7FFFFFFFull) return GEMM_ERR_INVALID_ARG;
  return launch_grouped<CG, OP, true, true, NT, OUT32>(tmP, tmQ, a, tiles, ctx, stream);
}

template <int CG, uint32_t NT>
int sum_pick(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
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
  // The pair's tiles of 256 x 256 where there are enough of them for every
  // pair and the MMAs, not the store, bound the call; one CTA's of 128 x 128
  // else.  Measured, us, one CTA / pair: 16 groups of 1040 x 2056, 256 rows
  // each, bf16 36.8 / 31.3, fp32 43.2 / 40.5; 64 rows each, bf16 25.1 / 24.1,
  // fp32 29.4 / 33.1; 8 groups of 512 x 512, 1024 rows each, bf16 8.8 / 12.5.
  const uint64_t tiles = ceil_div_u64(p.K, 256) * ceil_div_u64(p.N, 256) * p.groups;
  const bool pair = tiles >= static_cast<uint64_t>(ctx.num_sms / 2) &&
                    (!p.out_f32 || p.M / p.groups >= 256);
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
