// Decode kernels with scores kept for the weights for an fp16 cache.
#include "pkv_decode_impl.cuh"

namespace pkv {
cudaError_t launch_decode_scored_f16(const DecodeLaunch& l) {
  if (l.q_bf16 != false) return cudaErrorNotSupported;
  return dispatch_split<kCacheF16, false, kModeScored>(l);
}
}  // namespace pkv
