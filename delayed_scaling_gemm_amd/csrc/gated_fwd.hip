// Forward product of a gated feed-forward block: X times gate and up projections, activation and
// product in one kernel (gated.h).
#include "gated_launch.h"

namespace fp8ds {

hipError_t launch_gated_fwd(const GatedProblem& q, bool exact, int num_cus, hipStream_t stream) {
  if (q.M <= kGatedFewRows) return launch_gated_few(q, stream);
  return exact ? launch_gated_path<kE4M3, true, kEpiGate>(q, num_cus, stream)
               : launch_gated_path<kE4M3, false, kEpiGate>(q, num_cus, stream);
}

}  // namespace fp8ds
