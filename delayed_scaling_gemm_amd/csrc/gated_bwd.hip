// Backward product of a gated feed-forward block: dY times the down projection, through the
// activation, to the gradients of gate and up (gated.h).
#include "gated_launch.h"

namespace fp8ds {

hipError_t launch_gated_bwd(const GatedProblem& q, int fa, bool exact, int num_cus, hipStream_t stream) {
  if (fa == kE5M2)
    return exact ? launch_gated_path<kE5M2, true, kEpiGateBwd>(q, num_cus, stream)
                 : launch_gated_path<kE5M2, false, kEpiGateBwd>(q, num_cus, stream);
  return exact ? launch_gated_path<kE4M3, true, kEpiGateBwd>(q, num_cus, stream)
               : launch_gated_path<kE4M3, false, kEpiGateBwd>(q, num_cus, stream);
}

}  // namespace fp8ds
