// Paged prefill attention with capped scores, alone or with a distance bias.
#include "pkv_prefill_biased.cuh"

namespace pkv {
cudaError_t launch_prefill_cap(const PrefillLaunch& l) {
  if (l.p.slopes != nullptr) return pfb::launch_bias<kBiasCap | kBiasDist>(l);
  return pfb::launch_bias<kBiasCap>(l);
}
}  // namespace pkv
