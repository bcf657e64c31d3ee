// Paged prefill attention with capped scores, alone or with a distance bias.
#include "pkv_prefill.cuh"

namespace pkv {
cudaError_t launch_prefill_cap(const PrefillLaunch& l) {
  if (l.p.slopes != nullptr) return pf::launch_prefill_bias<kBiasCap | kBiasDist>(l);
  return pf::launch_prefill_bias<kBiasCap>(l);
}
}  // namespace pkv
