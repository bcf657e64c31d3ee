// Acceptance of a path through a tree of drafted tokens: the accepted tokens'
// K and V rows move up behind the sequence's past.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

// One CTA per (sequence, KV head).  The rows of the path are all staged in shared
// memory (asynchronous copies of 16 bytes) before any is written, so a path may
// name its nodes in any order.  Bound by latency: length and path, table entry,
// row, one dependent load after the other; so CTAs are small and many share an SM
// (with the rows in registers, a CTA of 256 threads held room for the longest
// path and 256 sequences took 15.1 us).
constexpr int kAcceptThreads = 128;
static_assert(2 * kMaxPath <= kAcceptThreads, "a thread per step and per scale");

__global__ void __launch_bounds__(kAcceptThreads) accept_path_kernel(const AcceptParams p) {
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv, tid = threadIdx.x;
  extern __shared__ uint4 stage[];                // [max_path][K row, V row]
  __shared__ int32_t src_row[kMaxPath], dst_row[kMaxPath];  // of the pool; -1: nothing moves
  griddep_wait_then_trigger();
  const int node = tid < p.max_path ? p.path[(int64_t)b * p.max_path + tid] : 0;
  const int ctx = p.context_lens[b], len = p.path_lens[b];
  const int q0 = p.q_start[b], q1 = p.q_start[b + 1];
  const int n = q0 < 0 || q1 < q0 ? -1 : q1 - q0;
  if (ctx < 0 || ctx > p.MBS * kPageSize || n < 0 || n > ctx || len < 0 || len > n ||
      len > p.max_path) {
    if (h == 0 && tid == 0) report_error(p.err_word, PKV_ERR_BOUNDS);
    return;
  }
  const int base = ctx - n;
  if (h == 0 && tid == 0 && p.new_lens != nullptr) p.new_lens[b] = base + len;
  if (tid < len) {
    const int32_t* table = p.block_tables + (int64_t)b * p.MBS;
    int src = -1, dst = -1;
    if (node < 0 || node >= n) {
      report_error(p.err_word, PKV_ERR_BOUNDS);
    } else if (node != tid) {
      const int su = base + node, du = base + tid;
      const int sb = table[su / kPageSize], db = table[du / kPageSize];
      if (sb < 0 || sb >= p.NB || db < 0 || db >= p.NB) {
        report_error(p.err_word, PKV_ERR_BOUNDS);
      } else {  // the pool has less than 2^31 rows
        src = (sb * p.Hkv + h) * kPageSize + su % kPageSize;
        dst = (db * p.Hkv + h) * kPageSize + du % kPageSize;
      }
    }
    src_row[tid] = src;
    dst_row[tid] = dst;
  }
  __syncthreads();
  const int cpr = p.row_bytes >> 4, shift = cpr == 16 ? 5 : 4;  // pieces of a row: 8 or 16
  const int pieces = len << shift;
  for (int c = tid; c < pieces; c += kAcceptThreads) {
    const int src = src_row[c >> shift], piece = c & (2 * cpr - 1);
    if (src < 0) continue;
    const uint4* from = static_cast<const uint4*>(piece < cpr ? p.k_cache : p.v_cache) +
                        (int64_t)src * cpr + (piece & (cpr - 1));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(stage + c)), "l"(from)
                 : "memory");
  }
  // E4M3 with per-token scales: a row's two scales, K's then V's, lie 16 apart
  float scale = 0.f;
  const bool scaled = p.scales != nullptr && tid < 2 * len && src_row[tid >> 1] >= 0;
  auto at = [&](int row) -> int64_t {
    return (row / kPageSize * (int64_t)2 + (tid & 1)) * kPageSize + row % kPageSize;
  };
  if (scaled) scale = p.scales[at(src_row[tid >> 1])];
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();  // every row is read
  for (int c = tid; c < pieces; c += kAcceptThreads) {
    const int dst = dst_row[c >> shift], piece = c & (2 * cpr - 1);
    if (dst < 0) continue;
    static_cast<uint4*>(piece < cpr ? p.k_cache : p.v_cache)[(int64_t)dst * cpr +
                                                            (piece & (cpr - 1))] = stage[c];
  }
  if (scaled) p.scales[at(dst_row[tid >> 1])] = scale;
}

cudaError_t launch_accept_path(const AcceptParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)p.max_path * 2 * p.row_bytes;  // at most 32 KB
  return launch_dependent(accept_path_kernel, dim3((unsigned)(p.B * p.Hkv)), dim3(kAcceptThreads),
                          smem, stream, p);
}

}  // namespace pkv
