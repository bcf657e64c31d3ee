// pkv_hd.h -- index arithmetic that kernels and host code share.  Needs no CUDA.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif

namespace pkv {

// a / b for a >= 0, b > 0: a 32-bit division when both fit (the usual case;
// a 64-bit division is a long instruction sequence)
PKV_HD int64_t udiv64(int64_t a, int64_t b) {
  if ((((uint64_t)a | (uint64_t)b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

}  // namespace pkv
