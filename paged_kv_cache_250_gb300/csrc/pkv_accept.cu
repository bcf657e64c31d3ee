// Acceptance of a path through a tree of drafted tokens: the accepted tokens'
// K and V rows move up behind the sequence's past.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

// One CTA per (sequence, KV head).  The rows of the path, up to kMaxPath of
// them, are all read into registers before any is written, so a path may name
// its nodes in any order.  Bound by latency: length, path, table entry, row,
// one dependent load after the other.
constexpr int kAcceptThreads = 256;
constexpr int kMaxChunks = kMaxPath * 2 * 16;  // 16-byte pieces of K and V rows of 256 bytes
constexpr int kPer = kMaxChunks / kAcceptThreads;

__global__ void __launch_bounds__(kAcceptThreads) accept_path_kernel(const AcceptParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv, tid = threadIdx.x;
  __shared__ int32_t path[kMaxPath];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid < p.max_path) path[tid] = p.path[(int64_t)b * p.max_path + tid];
  const int ctx = p.context_lens[b], n = p.q_start[b + 1] - p.q_start[b], len = p.path_lens[b];
  __syncthreads();
  if (ctx < 0 || ctx > p.MBS * kPageSize || n < 0 || n > ctx || len < 0 || len > n ||
      len > p.max_path) {
    if (h == 0 && tid == 0) report_error(p.err_word, PKV_ERR_BOUNDS);
    return;
  }
  const int base = ctx - n;
  if (h == 0 && tid == 0 && p.new_lens != nullptr) p.new_lens[b] = base + len;
  const int32_t* table = p.block_tables + (int64_t)b * p.MBS;
  // row of the pool that position u of this KV head lies in, or -1
  auto row_of = [&](int u) -> int64_t {
    const int blk = table[u / kPageSize];
    if (blk < 0 || blk >= p.NB) {
      report_error(p.err_word, PKV_ERR_BOUNDS);
      return -1;
    }
    return ((int64_t)blk * p.Hkv + h) * kPageSize + u % kPageSize;
  };
  auto node_of = [&](int i) -> int {  // the node that step i takes, or -1: nothing moves
    const int node = path[i];
    if (node < 0 || node >= n) {
      report_error(p.err_word, PKV_ERR_BOUNDS);
      return -1;
    }
    return node == i ? -1 : node;
  };
  const int cpr = p.row_bytes >> 4;  // pieces of a row: 8 or 16
  uint4 data[kPer];
  int64_t to[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int c = tid + e * kAcceptThreads, i = c / (2 * cpr), piece = c - i * 2 * cpr;
    to[e] = -1;
    if (i >= len) continue;
    const int node = node_of(i);
    if (node < 0) continue;
    const int64_t src = row_of(base + node), dst = row_of(base + i);
    if (src < 0 || dst < 0) continue;
    const uint4* from = static_cast<const uint4*>(piece < cpr ? p.k_cache : p.v_cache);
    data[e] = from[src * cpr + piece % cpr];
    to[e] = dst * cpr + piece % cpr;
  }
  // E4M3 with per-token scales: a row's two scales, K's then V's, lie 16 apart
  float scale = 0.f;
  float* scale_to = nullptr;
  if (p.scales != nullptr && tid < 2 * len) {
    const int i = tid >> 1, node = node_of(i);
    if (node >= 0) {
      const int64_t src = row_of(base + node), dst = row_of(base + i);
      auto at = [&](int64_t row) -> int64_t {
        return (row / kPageSize * 2 + (tid & 1)) * kPageSize + row % kPageSize;
      };
      if (src >= 0 && dst >= 0) {
        scale = p.scales[at(src)];
        scale_to = p.scales + at(dst);
      }
    }
  }
  __syncthreads();  // every row is read
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    if (to[e] < 0) continue;
    const int c = tid + e * kAcceptThreads, piece = c % (2 * cpr);
    static_cast<uint4*>(piece < cpr ? p.k_cache : p.v_cache)[to[e]] = data[e];
  }
  if (scale_to != nullptr) *scale_to = scale;
}
static_assert(2 * kMaxPath <= kAcceptThreads, "a thread per scale");

cudaError_t launch_accept_path(const AcceptParams& p, cudaStream_t stream) {
  return launch_dependent(accept_path_kernel, dim3((unsigned)(p.B * p.Hkv)), dim3(kAcceptThreads),
                          0, stream, p);
}

}  // namespace pkv
