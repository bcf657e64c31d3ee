// Paged prefill attention with scores under a wide cap, alone or with a distance bias.
#include "pkv_prefill.cuh"

namespace pkv {
cudaError_t launch_prefill_cap_fine(const PrefillLaunch& l) {
  if (l.p.slopes != nullptr) return pf::launch_prefill_bias<kBiasCap | kBiasFine | kBiasDist>(l);
  return pf::launch_prefill_bias<kBiasCap | kBiasFine>(l);
}
}  // namespace pkv
