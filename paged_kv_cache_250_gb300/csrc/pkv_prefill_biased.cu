// Paged prefill attention with capped scores, a distance bias, or both.
#include "pkv_prefill.cuh"

namespace pkv {
cudaError_t launch_prefill_biased(const PrefillLaunch& l) {
  const bool cap = l.p.cap_log2 > 0.f, dist = l.p.slopes != nullptr;
  if (cap && dist) return pf::launch_prefill_bias<kBiasCap | kBiasDist>(l);
  if (cap) return pf::launch_prefill_bias<kBiasCap>(l);
  if (dist) return pf::launch_prefill_bias<kBiasDist>(l);
  return launch_prefill(l);
}
}  // namespace pkv
