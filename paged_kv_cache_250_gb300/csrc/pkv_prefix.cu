// Attention of a whole batch over a prefix that its sequences share, on the
// 5th-generation tensor cores, and the merge with the sequences' own parts.
//
// Every (sequence, query head) row of one KV head multiplies the same K and V
// blocks, so the prefix is a dense product of R = B g rows (g query heads per
// KV head) with 128-token blocks, each block read once per 256 rows instead
// of once per sequence.  Per row the kernel keeps the running maximum m and
// sum l of an online softmax and the unnormalised output o; the blocks are
// cut over S CTAs, each leaving its (m, l, o) as a partial, and
//   out = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M),   M = max_i m_i,
// over the prefix's partials and the row's own part (normalised, with its log2
// sum in the place of m and l = 1).
//
// One CTA per (pair of 128-row tiles, KV head, split), with fixed roles that
// hand over through mbarriers, as the prefill kernel's:
//   warps 0-3, 4-7  softmax of stream 0, 1: one row per thread, TMEM lane t;
//   warp 8          issues the MMAs; warp 9 the tensor copies.
// A stream is a row tile with its accumulator.  Two tiles of rows share every
// block (K and V double-buffered); with one tile left, both streams are that
// tile, stream t taking every second block in buffer t, so the tensor cores
// still work on one stream under the other's softmax.
//   S = Q K^T   tcgen05.mma M 128 x N 128 x K d from shared memory;
//   P           hi + lo 16-bit pairs over S in tensor memory (the weights keep
//               about 16 bits, as in the framework's other attention kernels);
//   O += P V    tcgen05.mma with A from tensor memory, twice per 16 tokens.
#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace px {

constexpr int kRows = 128, kTok = 128;  // rows of a tile, cached tokens of a block
constexpr int kPages = kTok / kPageSize;
constexpr int kThreads = 320;
constexpr uint32_t kHalf = 16384;  // 128 rows x 128 bytes: 64 d columns of a tile or block
constexpr int kBarQ = 0, kBarKFull = 1, kBarVFull = 3, kBarKFree = 5, kBarVFree = 7,
              kBarSFull = 9, kBarPFull = 11, kBarODone = 13, kNumBars = 15;
constexpr uint32_t kTmemCols = 512;  // S0/P0, S1/P1, then O0, O1
constexpr uint64_t kWaitNs = 1000000000ull;

template <int D>
struct Plan {
  static constexpr int NH = D / 64;
  static constexpr uint32_t kOffK = 2 * NH * kHalf;
  static constexpr uint32_t kOffV = 4 * NH * kHalf;
  static constexpr uint32_t kOffBar = 6 * NH * kHalf;
  static constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;  // TMEM base, abort, counts, max
  static constexpr size_t kSmem = 1024 + kOffMisc + 12 + 4 * kNumBars;
};
template <bool B>
struct Masked {
  static constexpr bool value = B;
};

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const PrefixParams p, const __grid_constant__ CUtensorMap tmq,
                  const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv) {
  using PL = Plan<D>;
  constexpr int NH = PL::NH;
  constexpr uint32_t kOffK = PL::kOffK, kOffV = PL::kOffV, kOffBar = PL::kOffBar,
                     kOffMisc = PL::kOffMisc;
  const int pair = blockIdx.x % p.pairs, split = blockIdx.x / p.pairs;
  const int h = blockIdx.y;
  const int G = p.Hq / p.Hkv;
  const int R = p.B * G;
  const bool two = (2 * pair + 1) * kRows < R;  // two tiles of rows, else two streams of one
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the kernel behind this one reads nothing that this one writes before its
  // own end, and everything earlier is complete: it may start
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * (uint32_t)i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(base_ptr + kOffMisc);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(base_ptr + kOffMisc + 4);
  int32_t* max_len = reinterpret_cast<int32_t*>(base_ptr + kOffMisc + 8);
  volatile int32_t* armed = reinterpret_cast<volatile int32_t*>(base_ptr + kOffMisc + 12);

  if (warp == 0) {
    tmem_alloc(base + kOffMisc, kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    *abort_flag = 0;
    *max_len = 0;
    for (int i = 0; i < kNumBars; ++i) {
      armed[i] = 0;
      mbar_init(bar(i), (i == kBarPFull || i == kBarPFull + 1) ? kRows / 32 : 1);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the positions any sequence sees of the prefix: rows of V behind them may
  // never have been written
  auto ctx_of = [&](int b) -> int {  // what a sequence sees; the suffix pass reports bad lengths
    const int c = p.context_lens[b];
    return c < 0 || c > p.MBS * kPageSize ? 0 : min(c, p.npb * kPageSize);
  };
  {
    int m = 0;
    for (int b = tid; b < p.B; b += kThreads) m = max(m, ctx_of(b));
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0 && m > 0) atomicMax(max_len, m);
  }
  __syncthreads();
  const int seen = *max_len;
  const int nblk_all = (seen + kTok - 1) / kTok;
  const int blk0 = (int)((int64_t)nblk_all * split / p.splits);
  const int nblk = (int)((int64_t)nblk_all * (split + 1) / p.splits) - blk0;
  // stream t's blocks: blk0 + i (two tiles) or blk0 + 2 i + t (one)
  auto count_of = [&](int t) -> int { return two ? nblk : (nblk + 1 - t) / 2; };
  auto block_of = [&](int t, int i) -> int { return blk0 + (two ? i : 2 * i + t); };
  auto buf_of = [&](int t, int i) -> int { return two ? i & 1 : t; };
  auto use_of = [&](int i) -> int { return two ? i >> 1 : i; };  // of the buffer

  auto wait = [&](int i, uint32_t parity) -> bool {
    if (*abort_flag) return false;
    if (mbar_wait_bounded(bar(i), parity, kWaitNs)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp == 9) {
    // ------------------------------------------------------------ copies
    if (nblk > 0) {
      if (lane == 0) {
        armed[kBarQ] = 1;
        const int nq = two ? 2 : 1;
        mbar_arrive_expect_tx(bar(kBarQ), (uint32_t)nq * NH * kHalf);
        for (int t = 0; t < nq; ++t)
          for (int c = 0; c < NH; ++c)
            tma_load_3d(base + (uint32_t)(t * NH + c) * kHalf, &tmq, bar(kBarQ), c * 64, h * G,
                        (2 * pair + t) * (kRows / G));
      }
      const int streams = two ? 1 : 2;
      auto entry = [&](int t, int i) -> int {  // lane l < 8: page l's block
        const int pg = block_of(t, i) * kPages + lane;
        return lane < kPages && i < count_of(t) && pg < p.npb ? p.prefix_blocks[pg] : 0;
      };
      int cur[2] = {entry(0, 0), two ? 0 : entry(1, 0)};
      bool ok = true;
      for (int i = 0; ok && i < count_of(0); ++i) {
        const int nxt[2] = {entry(0, i + 1), two ? 0 : entry(1, i + 1)};
        for (int v = 0; ok && v < 2; ++v) {  // K of the streams, then V
          for (int t = 0; t < streams; ++t) {
            if (i >= count_of(t)) continue;
            const int j = block_of(t, i), bb = buf_of(t, i), u = use_of(i);
            const int npg = min(kPages, p.npb - j * kPages);
            int blk = t == 0 ? cur[0] : cur[1];
            if (lane < npg && (blk < 0 || blk >= p.NB)) {  // read as zeros, past the pool
              if (v == 0) report_error(p.err_word, PKV_ERR_BOUNDS);
              blk = p.NB;
            }
            const int full = (v ? kBarVFull : kBarKFull) + bb;
            if (u > 0)
              ok = __all_sync(0xffffffffu,
                              wait((v ? kBarVFree : kBarKFree) + bb, (uint32_t)((u - 1) & 1)));
            if (!ok) break;
            if (lane == 0) {
              armed[full] = armed[full] + 1;
              mbar_arrive_expect_tx(bar(full), (uint32_t)npg * NH * kPageSize * 128);
            }
            __syncwarp();
            if (lane < npg) {
              const uint32_t dst = base + (v ? kOffV : kOffK) + (uint32_t)bb * NH * kHalf +
                                   (uint32_t)lane * kPageSize * 128;
              const int r = (blk * p.Hkv + h) * kPageSize;
              for (int c = 0; c < NH; ++c)
                tma_load_2d_plain(dst + (uint32_t)c * kHalf,
                                  v ? (const void*)&tmv : (const void*)&tmk, bar(full), c * 64, r);
            }
          }
        }
        ok = ok && !__any_sync(0xffffffffu, *abort_flag != 0);
        cur[0] = nxt[0];
        cur[1] = nxt[1];
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMAs
    if (lane == 0 && nblk > 0) {
      constexpr uint32_t kIdS = idesc_f16(BF16, false, kRows, kTok);
      constexpr uint32_t kIdO = idesc_f16(BF16, true, kRows, D);
      auto commit = [&](int i) {
        armed[i] = armed[i] + 1;
        umma_commit(bar(i));
      };
      const uint64_t dq = sdesc(base, 16, 1024);
      const uint64_t dk = sdesc(base + kOffK, 16, 1024);
      const uint64_t dv = sdesc(base + kOffV, kHalf, 1024);
      auto qk = [&](int t, int i) {
        const uint64_t a0 = dq + ((uint64_t)(two ? t : 0) * NH * kHalf >> 4);
        const uint64_t b0 = dk + ((uint64_t)buf_of(t, i) * NH * kHalf >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (uint32_t)(ks >> 2) * kHalf + (uint32_t)(ks & 3) * 32;
          umma(tmem + (uint32_t)t * kTok, a0 + (off >> 4), b0 + (off >> 4), kIdS, ks > 0);
        }
        commit(kBarSFull + t);
        if (!two || t == 1) commit(kBarKFree + buf_of(t, i));
      };
      auto pv = [&](int t, int i) {  // P_t: per 64 tokens 32 columns of hi, then 32 of lo pairs
        const uint64_t b0 = dv + ((uint64_t)buf_of(t, i) * NH * kHalf >> 4);
        const uint32_t pt = tmem + (uint32_t)t * kTok;
        const uint32_t dt = tmem + 256 + (uint32_t)t * D;
#pragma unroll
        for (int ks = 0; ks < kTok / 16; ++ks) {
          const uint64_t bv = b0 + ((uint32_t)ks * 16 * 128 >> 4);
          const uint32_t pa = pt + (uint32_t)(ks >> 2) * 64 + (uint32_t)(ks & 3) * 8;
          umma_ts(dt, pa, bv, kIdO, i > 0 || ks > 0);
          umma_ts(dt, pa + 32, bv, kIdO, 1);
        }
        commit(kBarODone + t);
        if (!two || t == 1) commit(kBarVFree + buf_of(t, i));
      };
      bool ok = wait(kBarQ, 0);
      for (int t = 0; ok && t < 2; ++t) {
        if (count_of(t) == 0) continue;
        ok = wait(kBarKFull + buf_of(t, 0), 0);
        if (!ok) break;
        tc_fence_after();
        qk(t, 0);
      }
      for (int i = 0; ok && i < count_of(0); ++i) {
        for (int t = 0; ok && t < 2; ++t) {
          if (i >= count_of(t)) continue;
          ok = wait(kBarPFull + t, (uint32_t)(i & 1)) &&
               wait(kBarVFull + buf_of(t, i), (uint32_t)(use_of(i) & 1));
          if (!ok) break;
          tc_fence_after();
          pv(t, i);
          if (i + 1 < count_of(t)) {
            ok = wait(kBarKFull + buf_of(t, i + 1), (uint32_t)(use_of(i + 1) & 1));
            if (!ok) break;
            qk(t, i + 1);
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;           // stream
    const int tt = tid - t * kRows;    // row in the tile
    const int nt = count_of(t);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + (uint32_t)t * kTok + lane_base;
    const uint32_t t_o = tmem + 256 + (uint32_t)t * D + lane_base;
    const int row = (2 * pair + (two ? t : 0)) * kRows + tt;
    const int b = row / G;
    // last position the row sees; rows past the batch (zero q) see all, unused
    const int vis = (b < p.B ? ctx_of(b) : seen) - 1;
    const int all_vis = __reduce_min_sync(0xffffffffu, vis);
    const float c2 = p.scale_log2;
    float m_ref = -INFINITY, l_sum = 0.f;
    bool ok = true;
    uint32_t r[32];
    for (int i = 0; i < nt; ++i) {
      ok = __all_sync(0xffffffffu, wait(kBarSFull + t, (uint32_t)(i & 1)));
      if (!ok) break;
      tc_fence_after();
      const int tok0 = block_of(t, i) * kTok;
      const bool full = tok0 + kTok - 1 <= all_vis;
      uint32_t sa[32], sb[32];
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto qmax = [&](auto mc, const uint32_t (&sq)[32], int qq) {
        const int t0 = tok0 + 32 * qq;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float a = __uint_as_float(sq[2 * e]), c = __uint_as_float(sq[2 * e + 1]);
          if constexpr (decltype(mc)::value) {
            if (t0 + 2 * e > vis) a = -INFINITY;
            if (t0 + 2 * e + 1 > vis) c = -INFINITY;
          }
          m4[e & 3] = max3(m4[e & 3], a, c);
        }
      };
      // quarters 3, 2, 1, 0: quarter 0 is still in sb when the P pass starts
      auto max_pass = [&](auto mc) {
        tmem_ld32_issue(t_s + 96, sa);
        tmem_ld_wait(sa);
        tmem_ld32_issue(t_s + 64, sb);
        qmax(mc, sa, 3);
        tmem_ld_wait(sb);
        tmem_ld32_issue(t_s + 32, sa);
        qmax(mc, sb, 2);
        tmem_ld_wait(sa);
        tmem_ld32_issue(t_s + 0, sb);
        qmax(mc, sa, 1);
        tmem_ld_wait(sb);
        qmax(mc, sb, 0);
      };
      if (full) max_pass(Masked<false>{});
      else max_pass(Masked<true>{});
      const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c2;
      const bool grow = mx > m_ref + 8.f;  // lazy rescale, as in the prefill kernel
      float alpha = 1.f;
      if (grow) {
        alpha = ex2(m_ref - mx);
        m_ref = mx;
        l_sum *= alpha;
      }
      if (i > 0) {
        ok = __all_sync(0xffffffffu, wait(kBarODone + t, (uint32_t)((i - 1) & 1)));
        if (!ok) break;
        tc_fence_after();
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            tmem_ld32(t_o + (uint32_t)cc * 32, r);
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st32(t_o + (uint32_t)cc * 32, r);
          }
        }
      }
      const float mu = m_ref == -INFINITY ? 0.f : m_ref;
      const uint64_t c2x2 = f2(c2, c2), nmu2 = f2(-mu, -mu);
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
      uint32_t hi[16], lo[16];
      auto qp = [&](auto mc, const uint32_t (&sq)[32], int qq) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 y = f2_split(fma2(f2(__uint_as_float(sq[2 * e]),
                                            __uint_as_float(sq[2 * e + 1])), c2x2, nmu2));
          float p0 = ex2(y.x), p1 = ex2(y.y);
          if constexpr (decltype(mc)::value) {
            const int tk = tok0 + 32 * qq + 2 * e;
            if (tk > vis) p0 = 0.f;
            if (tk + 1 > vis) p1 = 0.f;
          }
          const uint64_t pp = f2(p0, p1);
          acc[e & 3] = add2(acc[e & 3], pp);
          hi[e] = pack2<BF16>(p0, p1);
          const float2 hf = unpack2<BF16>(hi[e]);
          const float2 l = f2_split(sub2(pp, f2(hf.x, hf.y)));
          lo[e] = pack2<BF16>(l.x, l.y);
        }
      };
      auto qst = [&](int qq) {
        const uint32_t c = (uint32_t)(64 * (qq >> 1) + 16 * (qq & 1));
        tmem_st16_issue(t_s + c, hi);
        tmem_st16_issue(t_s + c + 32, lo);
      };
      auto p_pass = [&](auto mc) {
        tmem_ld32_issue(t_s + 32, sa);
        qp(mc, sb, 0);
        tmem_ld_wait(sa);
        qst(0);
        tmem_ld32_issue(t_s + 64, sb);
        qp(mc, sa, 1);
        tmem_ld_wait(sb);
        qst(1);
        tmem_ld32_issue(t_s + 96, sa);
        qp(mc, sb, 2);
        tmem_ld_wait(sa);
        qst(2);
        qp(mc, sa, 3);
        qst(3);
      };
      if (full) p_pass(Masked<false>{});
      else p_pass(Masked<true>{});
      tmem_st_wait();
      {
        const float2 a0 = f2_split(add2(acc[0], acc[1])), a1 = f2_split(add2(acc[2], acc[3]));
        l_sum += (a0.x + a0.y) + (a1.x + a1.y);
      }
      // V rows that no sequence sees may hold anything (0 x NaN): zeroed in the
      // staged block by the stream that uses it first
      if (tok0 + kTok > seen && (t == 0 || !two)) {
        const int bb = buf_of(t, i);
        ok = __all_sync(0xffffffffu, wait(kBarVFull + bb, (uint32_t)(use_of(i) & 1)));
        if (!ok) break;
        const int first = max(0, seen - tok0);
        const uint32_t vb = base + kOffV + (uint32_t)bb * NH * kHalf;
        for (int e = tt; e < (kTok - first) * 8 * NH; e += kRows) {
          const int rr = first + e / (8 * NH), ch = e % (8 * NH);
          const uint32_t a = vb + (uint32_t)(ch >> 3) * kHalf + (uint32_t)rr * 128 +
                             (uint32_t)(ch & 7) * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarPFull + t));
    }
    // ---- the stream's partial: m, l and the unnormalised o of its rows
    if (ok && nt > 0) ok = __all_sync(0xffffffffu, wait(kBarODone + t, (uint32_t)((nt - 1) & 1)));
    const int64_t slot = ((int64_t)(h * p.pairs + pair) * 2) * p.splits +
                         (two ? t * p.splits + split : 2 * split + t);
    if (b < p.B) {
      const bool any = ok && nt > 0 && l_sum != 0.f;  // NaN counts: it has to show
      reinterpret_cast<float2*>(p.part_ml)[slot * kRows + tt] =
          any ? make_float2(m_ref, l_sum) : make_float2(-INFINITY, 0.f);
    }
    if (ok && nt > 0) {
      tc_fence_after();
      float* po = p.part_o + (slot * kRows + tt) * D;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        tmem_ld32(t_o + (uint32_t)cc * 32, r);
        if (b < p.B) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reinterpret_cast<float4*>(po + cc * 32)[e] =
                make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                            __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // let copies and MMAs in flight land before the memory is given back
    if (tid == 0) report_error(p.err_word, PKV_ERR_TIMEOUT);
    if (tid < kNumBars && tid != kBarPFull && tid != kBarPFull + 1 && armed[tid] > 0)
      mbar_wait_bounded(bar(tid), (uint32_t)((armed[tid] - 1) & 1), kWaitNs);
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- the merge: one CTA of kMergeWarps warps per row; a warp's 32 lanes hold
// the row's d columns (two or four each) and take every kMergeWarps-th partial
constexpr int kMergeWarps = 4;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) prefix_merge_kernel(const PrefixMergeParams p) {
  constexpr int V = D / 32;  // columns per lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t orow = blockIdx.x;  // b Hq + hq
  const int b = (int)(orow / p.Hq), hq = (int)(orow - (int64_t)b * p.Hq);
  const int G = p.Hq / p.Hkv, h = hq / G;
  const int row = b * G + hq - h * G, tile = row >> 7, pair = tile >> 1;
  const bool two = (2 * pair + 1) * kRows < p.B * G;
  const int n = two ? p.splits : 2 * p.splits;
  const int64_t slot0 = ((int64_t)(h * p.pairs + pair) * 2) * p.splits +
                        (two ? (tile & 1) * p.splits : 0);
  const int rr = row & 127;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + slot0 * kRows + rr;
  const float* po = p.part_o + (slot0 * kRows + rr) * D + lane * V;

  // the common maximum over all parts (every warp for itself)
  const float lse = p.lse[orow];  // the row's own part: log2 of its sum
  float M = lse;
  for (int k = lane; k < n; k += 32) M = fmaxf(M, ml[(int64_t)k * kRows].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float l = 0.f, acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  if (M == -INFINITY) M = 0.f;  // nothing at all, or nothing but NaN
  {
#pragma unroll 4
    for (int k = warp; k < n; k += kMergeWarps) {
      const float2 v = ml[(int64_t)k * kRows];
      if (v.y != 0.f) {  // a part with nothing in it was not written
        const float w = ex2(v.x - M);
        l += w * v.y;
        const float* x = po + (int64_t)k * kRows * D;
        if constexpr (V == 4) {
          const float4 o = *reinterpret_cast<const float4*>(x);
          acc[0] += w * o.x;
          acc[1] += w * o.y;
          acc[2] += w * o.z;
          acc[3] += w * o.w;
        } else {
          const float2 o = *reinterpret_cast<const float2*>(x);
          acc[0] += w * o.x;
          acc[1] += w * o.y;
        }
      }
    }
    if (warp == 0 && lse != -INFINITY) {
      const float w = ex2(lse - M);
      l += w;
      const float* x = p.own_o + orow * D + lane * V;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += w * x[e];
    }
  }
  __shared__ float sh[kMergeWarps][D + 1];
#pragma unroll
  for (int e = 0; e < V; ++e) sh[warp][lane * V + e] = acc[e];
  if (lane == 0) sh[warp][D] = l;
  __syncthreads();
  if (threadIdx.x >= D) return;
  float o = 0.f, sum = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    o += sh[w][threadIdx.x];
    sum += sh[w][D];
  }
  o = sum != 0.f ? o / sum : 0.f;
  const int64_t at = orow * D + threadIdx.x;
  if (p.out_dtype == PKV_F32) static_cast<float*>(p.out)[at] = o;
  else if (p.out_dtype == PKV_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
  else static_cast<__half*>(p.out)[at] = __float2half_rn(o);
}

template <bool BF16, int D>
cudaError_t launch(const PrefixLaunch& l) {
  auto kern = prefix_kernel<BF16, D>;
  constexpr size_t smem = Plan<D>::kSmem;
  static std::atomic<uint64_t> configured{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(l.p.pairs * l.p.splits), (unsigned)l.p.Hkv, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, l.p, l.tmap_q, l.tmap_k, l.tmap_v);
}

}  // namespace px

cudaError_t launch_prefix(const PrefixLaunch& l) {
  if (l.d == 64) return l.bf16 ? px::launch<true, 64>(l) : px::launch<false, 64>(l);
  if (l.d == 128) return l.bf16 ? px::launch<true, 128>(l) : px::launch<false, 128>(l);
  return cudaErrorNotSupported;
}

cudaError_t launch_prefix_merge(const PrefixMergeParams& p, int d, cudaStream_t stream) {
  auto kern = d == 64 ? px::prefix_merge_kernel<64> : px::prefix_merge_kernel<128>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.Hq), 1, 1);
  cfg.blockDim = dim3(px::kMergeWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace pkv
