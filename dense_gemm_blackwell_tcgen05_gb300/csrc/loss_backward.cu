// The losses' backward products over the logits (loss_kernels.cuh).
#include "launch_loss.cuh"

namespace gb300 {

int launch_loss_logits_backward(const LossOperands& o, const LossArgs& a, const LaunchCtx& ctx, cudaStream_t stream) {
  if (a.K > 64 * loss_segment(loss_tiles(a.M, a.N, a.K).cg, true))
    return a.ids != nullptr ? loss_pick<true, true, true>(o, a, ctx, nullptr, stream)
                            : loss_pick<true, false, true>(o, a, ctx, nullptr, stream);
  return a.ids != nullptr ? loss_pick<true, true, false>(o, a, ctx, nullptr, stream)
                          : loss_pick<true, false, false>(o, a, ctx, nullptr, stream);
}

}  // namespace gb300
