// Decode kernels with scores kept for the weights for a bf16 cache.
#include "pkv_decode_impl.cuh"

namespace pkv {
cudaError_t launch_decode_scored_bf16(const DecodeLaunch& l) {
  if (l.q_bf16 != true) return cudaErrorNotSupported;
  return dispatch_split<kCacheBF16, true, kModeScored>(l);
}
}  // namespace pkv
