// Decode kernels with capped scores for an fp16 cache.
#include "pkv_decode_impl.cuh"

namespace pkv {
cudaError_t launch_decode_cap_f16(const DecodeLaunch& l) {
  if (l.q_bf16 != false) return cudaErrorNotSupported;
  return dispatch_split<kCacheF16, false, kModeCap>(l);
}
}  // namespace pkv
