// The weights of a scored decode call: what each cached row received of its
// KV head's attention, added to what it received before.
//
// The decode kernel leaves every score x (log2 units) and, per query head, the
// logarithm of the row's sum (lse = m + log2 l).  A row's new weight is
//   w = decay w + sum over the g query heads of the KV head of 2^(x - lse).
// Bound by latency, and by HBM for large batches: per row 4 g bytes of scores, part
// of them still in L2, and its weight read and written.  The call takes 57.6 us for 32
// sequences of up to 4096 tokens (the plain decode 50.7, the decode kernel alone in
// this form 51 and 1.5 for its stores), 235 for 64 of 8192 tokens in a per-token E4M3
// cache (202; 67 MB of scores).  Four rows per thread with wide loads made no difference
// to either, nor did dropping the scores' lines from L2 once read (231).
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kWeightThreads = 256;

template <int G>
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const WeightParams p) {
  const int seg = blockIdx.x / p.splits, sub = blockIdx.x - seg * p.splits;
  const int b = seg / p.Hkv, h = seg - b * p.Hkv;
  griddep_wait_then_trigger();
  const int ctx = p.context_lens[b];
  if (ctx < 0 || ctx > p.MBS * kPageSize) return;  // reported by the decode kernel
  float lse[G];
#pragma unroll
  for (int i = 0; i < G; ++i) lse[i] = p.lse[(int64_t)b * p.Hkv * G + h * G + i];
  const float* scores = p.scores + (int64_t)seg * p.MBS * kPageSize * G;
  const int32_t* table = p.block_tables + (int64_t)b * p.MBS;
  for (int64_t u = (int64_t)sub * kWeightThreads + threadIdx.x; u < ctx;
       u += (int64_t)p.splits * kWeightThreads) {
    const int blk = table[u / kPageSize];
    if (blk < 0 || blk >= p.NB) continue;  // left out by the decode kernel, which reported it
    float* w = p.weights + ((int64_t)blk * p.Hkv + h) * kPageSize + u % kPageSize;
    const bool fresh = u == ctx - 1 || p.decay == 0.f;  // what is there means nothing
    const float old = fresh ? 0.f : *w;
    float x[G];
    const float* s = scores + u * G;
    if constexpr (G == 1) {
      x[0] = s[0];
    } else if constexpr (G == 2) {
      const float2 v = *reinterpret_cast<const float2*>(s);
      x[0] = v.x;
      x[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < G; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(s + i);
        x[i] = v.x;
        x[i + 1] = v.y;
        x[i + 2] = v.z;
        x[i + 3] = v.w;
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) sum += exp2f(x[i] - lse[i]);
    *w = fresh ? sum : fmaf(p.decay, old, sum);
  }
}

cudaError_t launch_weights(const WeightParams& p, int group, cudaStream_t stream) {
  auto kern = group == 1   ? weights_kernel<1>
              : group == 2 ? weights_kernel<2>
              : group == 4 ? weights_kernel<4>
                           : weights_kernel<8>;
  return launch_dependent(kern, dim3((unsigned)((int64_t)p.B * p.Hkv * p.splits)),
                          dim3(kWeightThreads), 0, stream, p);
}

}  // namespace pkv
