// Paged prefill attention with a distance bias.
#include "pkv_prefill_biased.cuh"

namespace pkv {
cudaError_t launch_prefill_dist(const PrefillLaunch& l) { return pfb::launch_bias<kBiasDist>(l); }
}  // namespace pkv
