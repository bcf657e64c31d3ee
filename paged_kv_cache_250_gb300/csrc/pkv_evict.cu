// Eviction by accumulated attention weight: of the rows that a sequence holds
// under a KV head, `budget` stay.
//
// Which.  A row's rank is an unsigned 32-bit key: guarded rows (the first
// positions and the most recent ones) above all others, those by weight (the
// float's bits, mapped so that they order as unsigned numbers; NaN above
// infinity), rows of a page outside the pool below all.  The budget-th largest
// key T is found digit by digit (8 bits each) from histograms; kept are
// the keys above T and, of those equal to T, the first by index, as many as
// the budget leaves.
//
// Where.  Kept rows below the budget stay where they are.  The rows below it
// that go are holes, and the i-th kept row behind the budget moves into the
// i-th hole: no more rows move than have to, sources and destinations never
// meet, and the order is the same on every run.  (A hole in a page outside the pool
// takes no row: the one that was to move there is lost, and the error reported.)
//
// One cluster of CL CTAs per (sequence, KV head), each with a contiguous slice
// of the rows: the keys stay in shared memory, a warp takes a contiguous stretch
// of them, so counts before a row are those of the CTAs, warps and lanes before.
// Histograms, counts and the two lists cross CTAs through distributed shared
// memory; CTA r then moves the pairs r, r + CL, ...
//
// Bound by latency: a chain of look-ups, histograms and counts, each a round of loads
// or a barrier, then one of moves; large prompts by HBM too.  Kernel alone, in a graph:
// 32 sequences that let one of 2049 rows go, 8 KV heads, 7 us; 64 that let 128 of 4224
// go 20 us (52 MB: its 512 CTAs run at once, 4 per SM); 8 prompts of up to 32768 rows
// cut to 4096 45 us, half of it the moves of 170 MB; one prompt of 131072 rows 28 us,
// on 64 SMs.  Digits of 11 bits (histograms of 8 KB, read by every CTA of a cluster
// from all others) took 161 us for the 8 prompts; several rows per thread in flight
// made no difference.
#include <cooperative_groups.h>

#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 256, kDigits = 4;
constexpr uint32_t kGuarded = 0xffffffffu, kNan = 0xfffffffeu;
constexpr int kMaxWarps = 32;
constexpr size_t kFixedSmem = kDigits * kBins * 4 + 2 * kMaxWarps * 4 + 32;
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
  return kFixedSmem + slice_rows(rows, cl) * 4 + slice_rows(rows, cl) / 4 +
         slice_rows(rows, cl) / kPageSize * 4;
}

template <int CL, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) evict_kernel(const EvictParams p) {
  constexpr int NW = NT / 32;
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* hist = smem;                       // [kDigits][kBins]
  uint32_t* warp_a = hist + kDigits * kBins;   // [NW] counts of the warps
  uint32_t* warp_b = warp_a + kMaxWarps;
  uint32_t* pick = warp_b + kMaxWarps;  // [4] digit, count above it, count in it
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
  for (int i = tid; i < kDigits * kBins; i += NT) hist[i] = 0;
  griddep_wait_then_trigger();
  const int n = p.context_lens[b], old = p.old_lens[b], told = p.num_tokens[b];
  if (n < 0 || n > p.MBS * kPageSize || old < 0 || old > n || told < n) {
    if (h == 0 && rank == 0 && tid == 0) report_error(p.err_word, PKV_ERR_BOUNDS);
    return;
  }
  if (h == 0 && rank == 0 && tid == 0) p.new_lens[b] = min(n, p.budget);
  const int slice = (int)slice_rows(n, CL);
  const int lo = (int)min((int64_t)n, (int64_t)rank * slice);
  const int cnt = min(slice, n - lo);          // rows lo .. lo + cnt - 1
  int* rows = reinterpret_cast<int*>(keys + slice);  // first row of each page, or -1
  uint8_t* nibs = reinterpret_cast<uint8_t*>(rows + slice / kPageSize);  // see below, four rows each
  const int32_t* table = p.block_tables + (int64_t)b * p.MBS;
  auto row_of = [&](int u) -> int {  // of the pool, or -1
    const int blk = table[u / kPageSize];
    if (blk < 0 || blk >= p.NB) return -1;
    return (blk * p.Hkv + h) * kPageSize + u % kPageSize;  // the pool has less than 2^31 rows
  };
  for (int i = tid; i < (cnt + kPageSize - 1) / kPageSize; i += NT) {
    rows[i] = row_of(lo + i * kPageSize);  // a slice is whole pages
    if (rows[i] < 0) report_error(p.err_word, PKV_ERR_BOUNDS);
  }
  __syncthreads();

  // ---- keys, and the positions of the rows that came since the last call; a
  // thread takes four rows of a page at a time
#pragma unroll 1
  for (int i = 4 * tid; i < cnt; i += 4 * NT) {
    const int u = lo + i, first = rows[i / kPageSize], row = first + i % kPageSize;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    int4 at = make_int4(0, 0, 0, 0);
    if (first >= 0 && n > p.budget) w = *reinterpret_cast<const float4*>(p.weights + row);
    if (first >= 0 && u < old) at = *reinterpret_cast<const int4*>(p.positions + row);
    const float wv[4] = {w.x, w.y, w.z, w.w};
    int pv[4] = {at.x, at.y, at.z, at.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (u + e >= old) pv[e] = told - n + u + e;
    if (first >= 0 && u >= old && i + 4 <= cnt) {
      *reinterpret_cast<int4*>(p.positions + row) = make_int4(pv[0], pv[1], pv[2], pv[3]);
    } else if (first >= 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (u + e >= old && i + e < cnt) p.positions[row + e] = pv[e];
    }
    if (n <= p.budget) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i + e >= cnt) break;
      uint32_t key = 0;
      if (first >= 0) key = pv[e] < p.sinks || pv[e] >= told - p.recent ? kGuarded : key_of(wv[e]);
      keys[i + e] = key;
      atomicAdd(&hist[key >> 24], 1u);
    }
  }
  if (n <= p.budget) return;  // the same in every CTA of the cluster
  sync();

  // ---- the budget-th largest key
  uint32_t T = 0, need = (uint32_t)p.budget;  // digits so far; rows still to keep
  uint32_t in_last = 0;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    uint32_t* hh = hist + (24 - shift) / 8 * kBins;
    if (shift < 24) {
      for (int i = 4 * tid; i < cnt; i += 4 * NT) {
        const uint4 k4 = *reinterpret_cast<const uint4*>(keys + i);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((k[e] ^ T) >> (shift + 8) == 0 && i + e < cnt)
            atomicAdd(&hh[(k[e] >> shift) & 0xff], 1u);
      }
      sync();
    }
    // thread t holds bin t counted from the highest
    uint32_t c = 0;
    if (tid < kBins) {
#pragma unroll
      for (int r = 0; r < CL; ++r) c += at_rank(hh, r)[kBins - 1 - tid];
    }
    uint32_t inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) warp_a[warp] = inc;
    __syncthreads();
    const uint32_t before =
        __reduce_add_sync(0xffffffffu, lane < warp ? warp_a[lane] : 0u) + inc - c;
    if (before < need && need <= before + c) {  // one thread
      pick[0] = (uint32_t)(kBins - 1 - tid);
      pick[1] = before;
      pick[2] = c;
    }
    __syncthreads();
    T |= pick[0] << shift;
    need -= pick[1];
    in_last = pick[2];
    if (need == in_last) break;  // every row whose key begins with these digits is kept
    __syncthreads();
  }
  // Kept are the keys above T and `need` of those that equal it.  (Where the
  // search ended early T is the least key that begins with the digits.)

  // ---- events: rows below the budget that go (holes), rows behind it that stay
  // (late rows).  A lane takes four rows of a warp's 128; a nibble says which of
  // them are events.
  const int per = (cnt + 128 * NW - 1) / (128 * NW) * 128;  // rows of a warp
  const int w0 = min(cnt, warp * per), w1 = min(cnt, w0 + per);
  auto lanes_before = [&](uint32_t v) -> uint32_t {  // sum over the lanes before this one
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x - v;
  };
  auto four = [&](int i, uint32_t (&k)[4]) -> uint32_t {  // keys i .. i + 3; those that equal T
    const uint4 v = i < w1 ? *reinterpret_cast<const uint4*>(keys + i) : make_uint4(0, 0, 0, 0);
    k[0] = v.x;
    k[1] = v.y;
    k[2] = v.z;
    k[3] = v.w;
    uint32_t eq = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) eq |= (i + e < w1 && k[e] == T ? 1u : 0u) << e;
    return eq;
  };
  __syncthreads();
  uint32_t ties = 0;  // rows with key T before this warp's
  if (need < in_last) {
    uint32_t k[4];
    for (int i = w0 + 4 * lane; i < w1; i += 128) ties += __popc(four(i, k));
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) warp_a[warp] = ties;
    __syncthreads();
    const uint32_t v = lane < NW ? warp_a[lane] : 0u;
    const uint32_t all = __reduce_add_sync(0xffffffffu, v);
    ties = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0u);
    if (tid == 0) tot[0] = all;
    sync();
    for (int r = 0; r < rank; ++r) ties += *at_rank(tot, r);
  }
  uint32_t events = 0, holes = 0;
  for (int i0 = w0; i0 < w1; i0 += 128) {
    const int i = i0 + 4 * lane, u = lo + i;
    uint32_t k[4], keep = 0;
    const uint32_t eq = four(i, k);
#pragma unroll
    for (int e = 0; e < 4; ++e) keep |= (k[e] >= T ? 1u : 0u) << e;
    if (need < in_last) {  // the first of the equal keys only
      uint32_t t = ties + lanes_before(__popc(eq));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((eq >> e) & 1)
          if (t++ >= need) keep &= ~(1u << e);
      ties += __reduce_add_sync(0xffffffffu, __popc(eq));
    }
    const uint32_t in = i >= w1 ? 0u : i + 4 <= w1 ? 15u : (1u << (w1 - i)) - 1;
    const uint32_t low = u >= p.budget ? 0u : u + 4 <= p.budget ? 15u : (1u << (p.budget - u)) - 1;
    const uint32_t ev = (keep ^ low) & in;
    if (in != 0) nibs[i >> 2] = (uint8_t)ev;
    events += __popc(ev);
    holes += __popc(ev & low);
  }
  events = __reduce_add_sync(0xffffffffu, events);
  holes = __reduce_add_sync(0xffffffffu, holes);
  __syncthreads();  // warp_a is free again
  if (lane == 0) {
    warp_a[warp] = events;
    warp_b[warp] = holes;
  }
  __syncthreads();
  const uint32_t ev_w = lane < NW ? warp_a[lane] : 0u;
  uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? ev_w : 0u);  // events before
  uint32_t pairs = __reduce_add_sync(0xffffffffu, lane < NW ? warp_b[lane] : 0u);
  if constexpr (CL > 1) {
    const uint32_t all = __reduce_add_sync(0xffffffffu, ev_w);
    if (tid == 0) {
      tot[1] = all;
      tot[2] = pairs;
    }
    sync();  // and the keys of every CTA are read for the last time
    pairs = 0;
    for (int r = 0; r < CL; ++r) {
      if (r < rank) at += at_rank(tot, r)[1];
      pairs += at_rank(tot, r)[2];
    }
  }

  // ---- the i-th hole and the i-th late row, over the keys: i / CL in the CTA
  // i % CL.  In the order of the rows all holes come before all late rows.  There
  // are at most n / 2 pairs, so both lists fit a slice.
  const int half = slice / 2;
  for (int i0 = w0; i0 < w1; i0 += 128) {
    const int i = i0 + 4 * lane;
    const uint32_t ev = i < w1 ? nibs[i >> 2] : 0u;
    uint32_t o = at + lanes_before(__popc(ev));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!((ev >> e) & 1)) continue;
      const uint32_t x = o < pairs ? o : o - pairs;
      at_rank(keys, (int)(x % CL))[(o < pairs ? 0 : half) + x / CL] = (uint32_t)(lo + i + e);
      ++o;
    }
    at += __reduce_add_sync(0xffffffffu, __popc(ev));
  }
  sync();
  int* to = reinterpret_cast<int*>(keys);
  int* from = to + half;
  const int mine = ((int)pairs - rank + CL - 1) / CL;

  // ---- the moves.  The lists become rows of the pool (-1: outside, nothing
  // moves); a thread takes the small things of a pair, whose loads are in flight
  // while K and V move.
#pragma unroll 1
  for (int i = tid; i < mine; i += NT) {
    const int u = from[i];
    int dst = row_of(to[i]), src = row_of(u);
    if (dst < 0 || src < 0) dst = src = -1;
    to[i] = dst;
    from[i] = src;
    if (src < 0) continue;
    const float w = p.weights[src];
    const int at = u >= old ? told - n + u : p.positions[src];
    if (p.scales != nullptr) {
      // a page's 16 K scales, then its 16 V scales
      const int64_t s0 = src + (int64_t)(src & ~(kPageSize - 1)), d0 = dst + (int64_t)(dst & ~(kPageSize - 1));
      const float k = p.scales[s0], v = p.scales[s0 + kPageSize];
      p.scales[d0] = k;
      p.scales[d0 + kPageSize] = v;
    }
    p.weights[dst] = w;
    p.positions[dst] = at;
  }
  __syncthreads();
  // K and V: 16 bytes per lane, a row's 2 cpr pieces side by side (a warp holds
  // one pair, or two of E4M3 and d 64), kAt steps in flight
  constexpr int kAt = 4;
  const int cpr = p.row_bytes >> 4;  // pieces of a row: 8 or 16
  const int wide = 16 / cpr;         // pairs per warp: 1 or 2
  const int sub = lane / (2 * cpr), piece = lane % (2 * cpr);
  const bool is_v = piece >= cpr;
  const uint4* in = static_cast<const uint4*>(is_v ? p.v_cache : p.k_cache) + piece % cpr;
  uint4* out = static_cast<uint4*>(is_v ? p.v_cache : p.k_cache) + piece % cpr;
  for (int i0 = warp * wide; i0 < mine; i0 += NW * wide * kAt) {
    uint4 data[kAt];
    int dst[kAt];
#pragma unroll
    for (int e = 0; e < kAt; ++e) {
      const int i = i0 + e * NW * wide + sub;
      dst[e] = i < mine ? to[i] : -1;
      if (dst[e] >= 0) data[e] = in[(int64_t)from[i] * cpr];
    }
#pragma unroll
    for (int e = 0; e < kAt; ++e)
      if (dst[e] >= 0) out[(int64_t)dst[e] * cpr] = data[e];
  }
}

}  // namespace

constexpr int kMaxCluster = 16;  // opt-in: more than the portable 8
constexpr int32_t kMaxBlocks = 49152;  // of a table: what the largest cluster holds
bool evict_fits(int32_t mbs) { return mbs <= kMaxBlocks; }
static_assert(smem_of((int64_t)kMaxBlocks * kPageSize, kMaxCluster) <= kSmemLimit, "fits");

template <int CL, int NT>
static cudaError_t launch_cluster(const EvictParams& p, cudaStream_t stream) {
  auto kern = evict_kernel<CL, NT>;
  static std::atomic<uint64_t> configured{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit);
    if (e == cudaSuccess && CL > 8)
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.Hkv * CL));
  cfg.blockDim = dim3(NT);
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

template <int CL>
static cudaError_t launch_threads(const EvictParams& p, int nt, cudaStream_t stream) {
  return nt == 1024  ? launch_cluster<CL, 1024>(p, stream)
         : nt == 512 ? launch_cluster<CL, 512>(p, stream)
                     : launch_cluster<CL, 256>(p, stream);
}

// A cluster's CTAs lie in one GPC, so clusters that hold one CTA per SM leave
// some SMs out: of this GPU's 152, 152, 76, 36, 15 and 7 clusters of 1 to 16 run
// at once (cudaOccupancyMaxActiveClusters).  A CTA has 1024 threads where all
// clusters run at once like that, 512 or 256 where two or four CTAs have to share
// an SM.  Clusters are as large as leaves every SM a CTA at most and a CTA 2048
// rows, and as few as hold the keys.
cudaError_t launch_evict(const EvictParams& p, int sms, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.MBS * kPageSize, segs = (int64_t)p.B * p.Hkv;
  auto at_once = [&](int cl) -> int64_t {
    return cl == 1 ? sms : cl == 2 ? sms / 2 : cl == 4 ? sms * 36 / 152 : cl == 8 ? sms / 10 : sms / 21;
  };
  int cl = 1;
  while (cl < kMaxCluster && (smem_of(rows, cl) > kSmemLimit ||
                              (segs <= at_once(2 * cl) && rows >= (int64_t)2 * cl * 2048)))
    cl *= 2;
  const int nt = segs <= at_once(cl) ? 1024 : segs <= 2 * at_once(cl) ? 512 : 256;
  switch (cl) {
    case 1: return launch_threads<1>(p, nt, stream);
    case 2: return launch_threads<2>(p, nt, stream);
    case 4: return launch_threads<4>(p, nt, stream);
    case 8: return launch_threads<8>(p, nt, stream);
    default: return launch_threads<16>(p, nt, stream);
  }
}

}  // namespace pkv
