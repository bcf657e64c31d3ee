// Decode attention for trees of drafted tokens, first form: one warp per (row,
// query head), the row's d elements over its lanes, one cached token after the
// other with a running maximum and sum.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace tr {

template <bool BF16, int D>
__global__ void tree_kernel(const TreeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y, j = blockIdx.x;
  const int hq = blockIdx.z * 4 + (threadIdx.x >> 5);
  if (hq >= p.Hq) return;
  const int s0 = p.q_start[b], n = p.q_start[b + 1] - s0, ctx = p.context_lens[b];
  if (s0 < 0 || n < 0 || n > p.max_q || s0 + n > p.total_q || ctx < n ||
      ctx > p.MBS * kPageSize) {
    if (lane == 0 && hq == 0 && j == 0) report_error(p.err_word, PKV_ERR_BOUNDS);
    return;
  }
  if (j >= n) return;
  const int64_t row = (int64_t)(s0 + j) * p.Hq + hq;
  const uint64_t mask = (uint64_t)p.tree_mask[s0 + j];
  const int h = hq / (p.Hq / p.Hkv);
  const uint16_t* qp = static_cast<const uint16_t*>(p.q) + row * D + lane * V;
  auto load = [](const uint16_t* x, float (&y)[V]) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 f = unpack2<BF16>(*reinterpret_cast<const uint32_t*>(x + e));
      y[e] = f.x;
      y[e + 1] = f.y;
    }
  };
  float q[V], o[V] = {}, m = -INFINITY, l = 0.f;
  load(qp, q);
  for (int u = 0; u < ctx; ++u) {
    if (u >= ctx - n && !((mask >> (u - (ctx - n))) & 1)) continue;
    const int blk = p.block_tables[(int64_t)b * p.MBS + u / kPageSize];
    if (blk < 0 || blk >= p.NB) {
      report_error(p.err_word, PKV_ERR_BOUNDS);
      continue;
    }
    const int64_t at = (((int64_t)blk * p.Hkv + h) * kPageSize + u % kPageSize) * D + lane * V;
    float k[V], v[V], s = 0.f;
    load(static_cast<const uint16_t*>(p.k_cache) + at, k);
    load(static_cast<const uint16_t*>(p.v_cache) + at, v);
#pragma unroll
    for (int e = 0; e < V; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o2);
    s *= p.scale_log2;
    const float nm = fmaxf(m, s), a = ex2(m - nm), w = ex2(s - nm);
    m = nm;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = o[e] * a + w * v[e];
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int64_t at = row * D + lane * V + e;
    const float x = o[e] * inv;
    if (p.out_dtype == PKV_F32) static_cast<float*>(p.out)[at] = x;
    else if (p.out_dtype == PKV_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(x);
    else static_cast<__half*>(p.out)[at] = __float2half_rn(x);
  }
}

}  // namespace tr

cudaError_t launch_tree(const TreeLaunch& l) {
  auto kern = l.p.d == 64 ? (l.bf16 ? tr::tree_kernel<true, 64> : tr::tree_kernel<false, 64>)
                          : (l.bf16 ? tr::tree_kernel<true, 128> : tr::tree_kernel<false, 128>);
  return launch_dependent(kern,
                          dim3((unsigned)l.p.max_q, (unsigned)l.p.B, (unsigned)((l.p.Hq + 3) / 4)),
                          dim3(128), 0, l.stream, l.p);
}

}  // namespace pkv
