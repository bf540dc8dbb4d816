// The losses' forward products over the logits (loss_kernels.cuh).
#include "launch_loss.cuh"

namespace gb300 {

int launch_loss_logits_forward(const LossOperands& o, LossArgs a, const LaunchCtx& ctx, uint32_t* slots,
                               cudaStream_t stream) {
  return a.ids != nullptr ? loss_pick<false, true, true>(o, a, ctx, slots, stream)
                          : loss_pick<false, false, true>(o, a, ctx, slots, stream);
}

}  // namespace gb300
