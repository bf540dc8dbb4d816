// Host-side launcher of loss_kernel: one-time set-up per kernel and device, the
// persistent grid, the choice of tiles.
#pragma once

#include <mutex>

#include "launch_grouped.cuh"
#include "loss_host.h"
#include "loss_kernels.cuh"

namespace gb300 {

// A launch's cluster and, for one that follows another kernel of its call, the
// programmatic dependency on it.
inline void loss_attributes(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int cg, bool chained) {
  unsigned n = 0;
  if (cg > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cg);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (chained) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
}

// Clusters of a kernel that run at once on the current device (found once, with
// the kernel's shared memory opted in).
template <class C, auto kern, int CG>
int loss_room(const LaunchCtx& ctx, uint64_t* room) {
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
    // (a split of the registers that asked for more than the launch's would be waited for without end)
    cudaFuncAttributes as_built = {};
    if (cudaFuncGetAttributes(&as_built, kern) != cudaSuccess || as_built.numRegs < static_cast<int>(C::kLeastRegs)) {
      cudaGetLastError();
      return GEMM_ERR_LAUNCH;
    }
    int clusters = ctx.num_sms / CG;
    if (CG > 1) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = CG;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(static_cast<unsigned>(CG) * static_cast<unsigned>(ctx.num_sms));
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

// Launches on min(tiles, room) clusters.  A launch over one block of rows writes a slot
// of partial results for each cluster, any other one for each tile of columns.
template <int CG, uint32_t NT, bool BACK, bool LIST, bool SEG>
int launch_loss(const LossOperands& o, LossArgs a, const LossTiles& tile, const LaunchCtx& ctx, uint32_t* slots,
                cudaStream_t stream) {
  using C = LossCfg<CG, NT, BACK, SEG>;
  const auto kern = loss_kernel<CG, NT, BACK, LIST, SEG>;
  uint64_t room = 0;
  if (const int rc = loss_room<C, loss_kernel<CG, NT, BACK, LIST, SEG>, CG>(ctx, &room); rc != GEMM_OK) return rc;
  CUtensorMap all, compact, q;
  if (!operand_map(&all, o.A, a.K, a.M, 1, o.lda, 0, C::P_BOX) || !operand_map(&q, o.B, a.K, a.N, 1, o.ldb, 0, tile.nt / CG))
    return GEMM_ERR_LAUNCH;
  compact = all;
  if (o.compact != nullptr && !operand_map(&compact, o.compact, a.K, a.M, 1, o.ld_compact, 0, C::P_BOX))
    return GEMM_ERR_LAUNCH;
  CUtensorMap out = all;
  a.boxes = C::kBoxes && (CG == 2 || a.M > 64);   // (loss_kernels.cuh: what either takes)
  if (a.boxes) {
    // (whole chunks of 32 columns: the pitch has room for them)
    const uint64_t dims[3] = {a.ld_out, o.out_rows, 1}, strides[2] = {2 * a.ld_out, 2 * a.ld_out};
    const uint32_t box[3] = {32, 32, 1};
    if (!encode_map_3d(&out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.out, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B))
      return GEMM_ERR_LAUNCH;
  }
  a.nt = tile.nt;
  const uint64_t blocks = ceil_div_u64(a.M, C::LT), columns = ceil_div_u64(a.N, a.nt);
  if (blocks > 0x7FFFFFFFull / columns) return GEMM_ERR_INVALID_ARG;
  const uint64_t tiles = blocks * columns;
  uint64_t clusters = tiles < room ? tiles : room;
  if (!BACK) {
    a.runs = blocks == 1 ? 1u : 0u;
    const uint64_t most = tile.slots(a.M, a.N);
    if (a.runs && clusters > most) clusters = most;
    *slots = static_cast<uint32_t>(a.runs ? clusters : columns);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * CG));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  loss_attributes(cfg, attr, CG, o.chained);
  a.status = ctx.status;
  a.timeout_ns = ctx.timeout_ns;
  note_schedule(cfg.gridDim.x / CG, CG, static_cast<uint32_t>(tiles), 0u, 0u, 0u, 0u);
  if (const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, all, compact, q, out, a); e != cudaSuccess) {
    note_cuda_error(e);
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

template <bool BACK, bool LIST, bool SEG>
int loss_pick(const LossOperands& o, const LossArgs& a, const LaunchCtx& ctx, uint32_t* slots, cudaStream_t stream) {
  const LossTiles t = loss_tiles(a.M, a.N, a.K);
  return t.cg == 2 ? launch_loss<2, 256, BACK, LIST, SEG>(o, a, t, ctx, slots, stream)
                   : launch_loss<1, 128, BACK, LIST, SEG>(o, a, t, ctx, slots, stream);
}

}  // namespace gb300
