// Grouped products that reduce over the grouped rows: the gradient to the
// weights (Op::Sum of grouped_kernels.cuh), and the fill of an empty reduction.
#include "launch_grouped.cuh"

namespace gb300 {
namespace {

template <bool OUT32>
int sum_impl(const GroupedProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  constexpr int CG = 1;
  constexpr uint32_t NT = 128;
  using C = GroupedCfg<CG, Op::Sum, true, true, NT, OUT32>;
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
  a.accumulate = p.accumulate ? 1u : 0u;
  a.fmt = 1;
  a.status = ctx.status;
  a.timeout_ns = ctx.timeout_ns;
  a.stall_iter = p.stall_iter;
  const uint64_t tiles = ceil_div_u64(p.K, C::LT) * ceil_div_u64(p.N, NT) * p.groups;
  if (tiles > 0x7FFFFFFFull) return GEMM_ERR_INVALID_ARG;
  return launch_grouped<CG, Op::Sum, true, true, NT, OUT32>(tmP, tmQ, a, tiles, ctx, stream);
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
  return p.out_f32 ? sum_impl<true>(p, ctx, stream) : sum_impl<false>(p, ctx, stream);
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
