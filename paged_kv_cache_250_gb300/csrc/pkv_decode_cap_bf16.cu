// Decode kernels with capped scores for a bf16 cache.
#include "pkv_decode_impl.cuh"

namespace pkv {
cudaError_t launch_decode_cap_bf16(const DecodeLaunch& l) {
  if (l.q_bf16 != true) return cudaErrorNotSupported;
  return dispatch_split<kCacheBF16, true, kModeCap>(l);
}
}  // namespace pkv
