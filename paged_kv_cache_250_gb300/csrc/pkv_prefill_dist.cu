// Paged prefill attention with a distance bias.
#include "pkv_prefill.cuh"

namespace pkv {
cudaError_t launch_prefill_dist(const PrefillLaunch& l) {
  return pf::launch_prefill_bias<kBiasDist>(l);
}
}  // namespace pkv
