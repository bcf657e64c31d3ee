// Decode kernels with a distance bias for an E4M3 (fp8) cache
// with per-head scales.
#include "pkv_decode_impl.cuh"

namespace pkv {
cudaError_t launch_decode_dist_e4m3(const DecodeLaunch& l) {
  return l.q_bf16 ? dispatch_split<kCacheE4M3, true, kModeDist>(l)
                  : dispatch_split<kCacheE4M3, false, kModeDist>(l);
}
}  // namespace pkv
