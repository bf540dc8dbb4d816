// Host-side launcher of grouped_kernel: one-time set-up per kernel and
// device, the persistent grid, the cluster and dependency attributes.
#pragma once

#include <mutex>

#include "gemm_gb300.h"
#include "gemm_host.h"
#include "grouped_host.h"
#include "grouped_kernels.cuh"

namespace gb300 {

// Tensor map of a batch of 16-bit matrices read in tiles of 64 elements along
// their contiguous dimension and box_rows rows, 128-byte swizzled.
inline bool operand_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows, uint64_t batch,
                        uint64_t ld, uint64_t stride, uint32_t box_rows) {
  // a single matrix's stride is never used; any legal value will do
  const uint64_t dims[3] = {inner, rows, batch};
  const uint64_t strides[2] = {ld * 2, (batch > 1 ? stride : ld) * 2};
  const uint32_t box[3] = {64, box_rows, 1};
  return encode_map_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, base, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

// Rows of the operand boxes of a kernel: 64 k rows of an MN-major operand;
// 128 rows of a K-major P, Q_BOX of a K-major Q.
template <class C, bool MN>
constexpr uint32_t p_box_rows() { return MN ? 64u : 128u; }
template <class C, bool MN>
constexpr uint32_t q_box_rows() { return MN ? 64u : C::Q_BOX; }

// Clusters of a kernel that run at once on the current device (found once, with
// the kernel's shared memory opted in).
template <int CG, Op OP, bool P_MN, bool Q_MN, uint32_t NT, bool OUT32, uint32_t SPLIT = 1>
int grouped_room(const LaunchCtx& ctx, uint64_t* room) {
  using C = GroupedCfg<CG, OP, P_MN, Q_MN, NT, OUT32, SPLIT>;
  const auto kern = grouped_kernel<CG, OP, P_MN, Q_MN, NT, OUT32, SPLIT>;
  static std::mutex mu;
  static int resident[128] = {0};   // per device (0: not set up yet)
  if (ctx.device < 0 || ctx.device >= 128) return GEMM_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lk(mu);
  if (resident[ctx.device] == 0) {
    if (const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(C::SMEM_BYTES));
        e != cudaSuccess) {
      note_cuda_error(e);
      cudaGetLastError();
      return GEMM_ERR_LAUNCH;
    }
    int clusters = ctx.num_sms / static_cast<int>(C::kCluster);
    if (C::kCluster > 1) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = C::kCluster;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(static_cast<unsigned>(C::kCluster) * static_cast<unsigned>(ctx.num_sms));
      cfg.blockDim = dim3(C::kThreads);
      cfg.dynamicSmemBytes = C::SMEM_BYTES;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int found = 0;
      if (cudaOccupancyMaxActiveClusters(&found, kern, &cfg) == cudaSuccess && found > 0) clusters = found;
      else cudaGetLastError();
    }
    resident[ctx.device] = clusters;
  }
  *room = static_cast<uint64_t>(resident[ctx.device]);
  return GEMM_OK;
}

// Launches on min(tiles, room) clusters.
template <int CG, Op OP, bool P_MN, bool Q_MN, uint32_t NT, bool OUT32, uint32_t SPLIT = 1>
int launch_grouped(const CUtensorMap& tmP, const CUtensorMap& tmQ, const GroupedArgs& a, uint64_t tiles,
                   const LaunchCtx& ctx, cudaStream_t stream) {
  using C = GroupedCfg<CG, OP, P_MN, Q_MN, NT, OUT32, SPLIT>;
  const auto kern = grouped_kernel<CG, OP, P_MN, Q_MN, NT, OUT32, SPLIT>;
  uint64_t room = 0;
  if (const int rc = grouped_room<CG, OP, P_MN, Q_MN, NT, OUT32, SPLIT>(ctx, &room); rc != GEMM_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((tiles < room ? tiles : room) * C::kCluster));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (C::kCluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = C::kCluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (a.pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  const uint32_t all = static_cast<uint32_t>(tiles), part = (a.K + C::BK - 1) / C::BK;
  note_schedule(cfg.gridDim.x / C::kCluster, C::kCluster, SPLIT > 1 ? 0u : all, SPLIT > 1 ? all : 0u,
                SPLIT > 1 ? (part + SPLIT - 1) / SPLIT : 0u, 0u, 0u);
  if (const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmP, tmQ, a); e != cudaSuccess) {
    note_cuda_error(e);
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

inline uint64_t ceil_div_u64(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

}  // namespace gb300
