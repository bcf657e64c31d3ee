// Eviction by accumulated attention weight: of the rows that a sequence holds
// under a KV head, `budget` stay.
//
// Which.  A row's rank is an unsigned 32-bit key: guarded rows (the first
// positions and the most recent ones) above all others, those by weight (the
// float's bits, mapped so that they order as unsigned numbers; NaN above
// infinity), rows of a page outside the pool below all.  The budget-th largest
// key T is found digit by digit (11, 11 and 10 bits) from histograms; kept are
// the keys above T and, of those equal to T, the first by index, as many as
// the budget leaves.
//
// Where.  Kept rows below the budget stay where they are.  The rows below it
// that go are holes, and the i-th kept row behind the budget moves into the
// i-th hole: no more rows move than have to, sources and destinations never
// meet, and the order is the same on every run.
//
// One cluster of CL CTAs per (sequence, KV head), each with a contiguous slice
// of the rows: the keys stay in shared memory, a warp takes a contiguous stretch
// of them, so counts before a row are those of the CTAs and warps before plus a
// ballot.  Histograms, counts and the two lists cross CTAs through distributed
// shared memory; CTA r then moves the pairs r, r + CL, ...
#include <cooperative_groups.h>

#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048;  // of a digit
constexpr uint32_t kGuarded = 0xffffffffu, kNan = 0xfffffffeu;
constexpr size_t kFixedSmem = 3 * kBins * 4 + 2 * kWarps * 4 + 32;
constexpr size_t kSmemLimit = 227 * 1024;

__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return kNan;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// rows of a CTA's slice: whole warps of 32
__host__ __device__ constexpr int64_t slice_rows(int64_t rows, int cl) {
  return (rows + 32 * cl - 1) / (32 * cl) * 32;
}
constexpr size_t smem_of(int64_t rows, int cl) {
  return kFixedSmem + slice_rows(rows, cl) * 4 + slice_rows(rows, cl) / 8;
}

template <int CL>
__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint32_t smem[];
  uint32_t* hist = smem;                // [3][kBins]
  uint32_t* warp_a = hist + 3 * kBins;  // [kWarps] counts of the warps
  uint32_t* warp_b = warp_a + kWarps;
  uint32_t* pick = warp_b + kWarps;     // [4] digit, count above it, count in it
  uint32_t* tot = pick + 4;             // [3] this CTA's ties, holes, late rows
  uint32_t* keys = tot + 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x / CL, rank = blockIdx.x - seg * CL;
  const int b = seg / p.Hkv, h = seg - b * p.Hkv;
  auto sync = [] {
    if constexpr (CL > 1) cg::this_cluster().sync();
    else __syncthreads();
  };
  auto at_rank = [](uint32_t* x, int r) -> uint32_t* {
    if constexpr (CL > 1) return cg::this_cluster().map_shared_rank(x, r);
    else return x;
  };
  for (int i = tid; i < 3 * kBins; i += kThreads) hist[i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = p.context_lens[b], old = p.old_lens[b], told = p.num_tokens[b];
  if (n < 0 || n > p.MBS * kPageSize || old < 0 || old > n || told < n) {
    if (h == 0 && rank == 0 && tid == 0) report_error(p.err_word, PKV_ERR_BOUNDS);
    return;
  }
  if (h == 0 && rank == 0 && tid == 0) p.new_lens[b] = min(n, p.budget);
  const int slice = (int)slice_rows(n, CL);
  const int lo = (int)min((int64_t)n, (int64_t)rank * slice);
  const int cnt = min(slice, n - lo);          // rows lo .. lo + cnt - 1
  uint32_t* bits = keys + slice;               // a bit per row: kept
  const int32_t* table = p.block_tables + (int64_t)b * p.MBS;
  auto row_of = [&](int u) -> int64_t {  // of the pool, or -1
    const int blk = table[u / kPageSize];
    if (blk < 0 || blk >= p.NB) return -1;
    return ((int64_t)blk * p.Hkv + h) * kPageSize + u % kPageSize;
  };
  __syncthreads();

  // ---- keys, and the positions of the rows that came since the last call
  for (int i = tid; i < cnt; i += kThreads) {
    const int u = lo + i;
    const int64_t row = row_of(u);
    uint32_t key = 0;
    if (row < 0) {
      report_error(p.err_word, PKV_ERR_BOUNDS);
    } else {
      const int pos = u >= old ? told - n + u : p.positions[row];
      if (u >= old) p.positions[row] = pos;
      key = pos < p.sinks || pos >= told - p.recent ? kGuarded : key_of(p.weights[row]);
    }
    if (n > p.budget) {
      keys[i] = key;
      atomicAdd(&hist[key >> 21], 1u);
    }
  }
  if (n <= p.budget) return;  // the same in every CTA of the cluster
  sync();

  // ---- the budget-th largest key
  uint32_t prefix = 0, need = (uint32_t)p.budget;  // digits so far; rows still to keep
  uint32_t in_last = 0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    uint32_t* hh = hist + pass * kBins;
    if (pass > 0) {
      for (int i = tid; i < cnt; i += kThreads) {
        const uint32_t k = keys[i];
        if (k >> (pass == 1 ? 21 : 10) == prefix)
          atomicAdd(&hh[(k >> shift) & (pass == 1 ? 0x7ff : 0x3ff)], 1u);
      }
      sync();
    }
    // thread t holds bins 2 t and 2 t + 1 counted from the highest
    const int top = kBins - 1 - 2 * tid;
    uint32_t c0 = 0, c1 = 0;
#pragma unroll
    for (int r = 0; r < CL; ++r) {
      const uint2 c = *reinterpret_cast<const uint2*>(at_rank(hh, r) + top - 1);
      c0 += c.y;
      c1 += c.x;
    }
    uint32_t inc = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) warp_a[warp] = inc;
    __syncthreads();
    const uint32_t before =
        __reduce_add_sync(0xffffffffu, lane < warp ? warp_a[lane] : 0u) + inc - c0 - c1;
    if (before < need && need <= before + c0 + c1) {  // one thread
      const bool second = need > before + c0;
      pick[0] = (uint32_t)(second ? top - 1 : top);
      pick[1] = second ? before + c0 : before;
      pick[2] = second ? c1 : c0;
    }
    __syncthreads();
    prefix = prefix << (pass == 2 ? 10 : 11) | pick[0];
    need -= pick[1];
    in_last = pick[2];
    __syncthreads();
  }
  const uint32_t T = prefix;  // `need` of the in_last rows with this key are kept

  // ---- kept rows, holes and late rows
  const int per = (cnt + 32 * kWarps - 1) / (32 * kWarps) * 32;  // rows of a warp
  const int w0 = min(cnt, warp * per), w1 = min(cnt, w0 + per);
  const uint32_t below = (1u << lane) - 1;
  uint32_t ties = 0;  // rows with key T before this warp's
  if (need < in_last) {
    for (int i0 = w0; i0 < w1; i0 += 32)
      ties += __popc(__ballot_sync(0xffffffffu, i0 + lane < w1 && keys[i0 + lane] == T));
    if (lane == 0) warp_a[warp] = ties;
    __syncthreads();
    const uint32_t all = __reduce_add_sync(0xffffffffu, warp_a[lane]);
    ties = __reduce_add_sync(0xffffffffu, lane < warp ? warp_a[lane] : 0u);
    if (tid == 0) tot[0] = all;
    sync();
    for (int r = 0; r < rank; ++r) ties += *at_rank(tot, r);
  }
  uint32_t holes = 0, late = 0;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < w1;
    const uint32_t k = in ? keys[i] : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, in && k == T);
    const bool keep = in && (k > T || (k == T && ties + __popc(eq & below) < need));
    if (need < in_last) ties += __popc(eq);
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    holes += __popc(__ballot_sync(0xffffffffu, in && !keep && lo + i < p.budget));
    late += __popc(__ballot_sync(0xffffffffu, keep && lo + i >= p.budget));
    if (lane == 0) bits[i0 >> 5] = kept;
  }
  __syncthreads();  // warp_a is free again
  if (lane == 0) {
    warp_a[warp] = holes;
    warp_b[warp] = late;
  }
  __syncthreads();
  const uint32_t hv = warp_a[lane], lv = warp_b[lane];
  int pairs = (int)__reduce_add_sync(0xffffffffu, hv);
  uint32_t hole_at = __reduce_add_sync(0xffffffffu, lane < warp ? hv : 0u);
  uint32_t late_at = __reduce_add_sync(0xffffffffu, lane < warp ? lv : 0u);
  if constexpr (CL > 1) {
    const uint32_t lates = __reduce_add_sync(0xffffffffu, lv);
    if (tid == 0) {
      tot[1] = (uint32_t)pairs;
      tot[2] = lates;
    }
    sync();  // and the keys of every CTA are read for the last time
    pairs = 0;
    for (int r = 0; r < CL; ++r) {
      const uint32_t hr = at_rank(tot, r)[1], lr = at_rank(tot, r)[2];
      if (r < rank) {
        hole_at += hr;
        late_at += lr;
      }
      pairs += (int)hr;
    }
  }

  // ---- the i-th hole and the i-th late row, over the keys: i / CL in the CTA
  // i % CL.  There are at most n / 2 pairs, so both lists fit a slice.
  const int half = slice / 2;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int u = lo + i0 + lane;
    const bool in = i0 + lane < w1, keep = (bits[i0 >> 5] >> lane) & 1;
    const bool is_hole = in && !keep && u < p.budget, is_late = keep && u >= p.budget;
    const uint32_t hb = __ballot_sync(0xffffffffu, is_hole);
    const uint32_t lb = __ballot_sync(0xffffffffu, is_late);
    if (is_hole) {
      const uint32_t i = hole_at + __popc(hb & below);
      at_rank(keys, (int)(i % CL))[i / CL] = (uint32_t)u;
    }
    if (is_late) {
      const uint32_t i = late_at + __popc(lb & below);
      at_rank(keys, (int)(i % CL))[half + i / CL] = (uint32_t)u;
    }
    hole_at += __popc(hb);
    late_at += __popc(lb);
  }
  sync();
  const uint32_t* from = keys + half;
  const int mine = (pairs - rank + CL - 1) / CL;

  // ---- the moves: a warp takes four pairs at a time, 16 bytes per lane
  constexpr int kAt = 4;
  const int cpr = p.row_bytes >> 4;  // pieces of a row: 8 or 16
  for (int i0 = warp * kAt; i0 < mine; i0 += kWarps * kAt) {
    // lane 2 i: the hole's row of pair i; lane 2 i + 1: the late row's
    int64_t row = -1;
    int at = 0;
    if (lane < 2 * kAt && i0 + (lane >> 1) < mine) {
      at = (int)(lane & 1 ? from[i0 + (lane >> 1)] : keys[i0 + (lane >> 1)]);
      row = row_of(at);
    }
    int64_t to[kAt], src[kAt];
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      to[i] = __shfl_sync(0xffffffffu, row, 2 * i);
      src[i] = __shfl_sync(0xffffffffu, row, 2 * i + 1);
    }
    const int late_u = __shfl_down_sync(0xffffffffu, at, 1);
    const int64_t late_row = __shfl_down_sync(0xffffffffu, row, 1);
    if (lane < 2 * kAt && !(lane & 1) && row >= 0 && late_row >= 0) {
      p.weights[row] = p.weights[late_row];
      p.positions[row] = late_u >= old ? told - n + late_u : p.positions[late_row];
      if (p.scales != nullptr) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          auto of = [&](int64_t r) { return (r / kPageSize * 2 + i) * kPageSize + r % kPageSize; };
          p.scales[of(row)] = p.scales[of(late_row)];
        }
      }
    }
    uint4 kv[kAt];
    bool go[kAt];
    // 16 pieces: half the lanes take K, the others V; 8: the lanes above 16 rest
    const int which = lane / cpr;
    const uint4* in = static_cast<const uint4*>(which == 0 ? p.k_cache : p.v_cache);
    uint4* out = static_cast<uint4*>(which == 0 ? p.k_cache : p.v_cache);
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      go[i] = which < 2 && to[i] >= 0 && src[i] >= 0;
      if (go[i]) kv[i] = in[src[i] * cpr + lane % cpr];
    }
#pragma unroll
    for (int i = 0; i < kAt; ++i)
      if (go[i]) out[to[i] * cpr + lane % cpr] = kv[i];
  }
}

}  // namespace

constexpr int kMaxCluster = 8;
constexpr int32_t kMaxBlocks = 24576;  // of a table: what the largest cluster holds
bool evict_fits(int32_t mbs) { return mbs <= kMaxBlocks; }

static_assert(smem_of((int64_t)kMaxBlocks * kPageSize, kMaxCluster) <= kSmemLimit, "fits");

template <int CL>
static cudaError_t launch_cluster(const EvictParams& p, cudaStream_t stream) {
  auto kern = evict_kernel<CL>;
  static std::atomic<uint64_t> configured{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.Hkv * CL));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_of((int64_t)p.MBS * kPageSize, CL);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_evict(const EvictParams& p, int sms, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.MBS * kPageSize, segs = (int64_t)p.B * p.Hkv;
  int cl = 1;
  while (cl < kMaxCluster && (smem_of(rows, cl) > kSmemLimit ||
                              (segs * 2 * cl <= sms && rows / (2 * cl) >= 2048)))
    cl *= 2;
  switch (cl) {
    case 1: return launch_cluster<1>(p, stream);
    case 2: return launch_cluster<2>(p, stream);
    case 4: return launch_cluster<4>(p, stream);
    default: return launch_cluster<8>(p, stream);
  }
}

}  // namespace pkv
