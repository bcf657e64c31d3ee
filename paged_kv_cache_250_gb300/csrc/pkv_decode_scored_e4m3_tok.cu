// Decode kernels with scores kept for the weights for an E4M3 (fp8) cache
// with per-token scales.
#include "pkv_decode_impl.cuh"

namespace pkv {
cudaError_t launch_decode_scored_e4m3_tok(const DecodeLaunch& l) {
  return l.q_bf16 ? dispatch_split<kCacheE4M3Tok, true, kModeScored>(l)
                  : dispatch_split<kCacheE4M3Tok, false, kModeScored>(l);
}
}  // namespace pkv
