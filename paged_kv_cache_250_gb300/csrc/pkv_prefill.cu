// Paged prefill attention: the kernels without a score bias (pkv_prefill.cuh).
#include "pkv_prefill.cuh"

namespace pkv {
cudaError_t launch_prefill(const PrefillLaunch& l) { return pf::launch_prefill_bias<0>(l); }
}  // namespace pkv
