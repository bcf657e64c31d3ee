// Decode attention of a batch whose sequences share a prefix: the prefix for
// the whole batch on the 5th-generation tensor cores, the sequences' own parts,
// and the merge.
//
// Every (sequence, query head) row of one KV head multiplies the same K and V
// blocks of the prefix, so it is a dense product of R = B g rows (g query heads
// per KV head) with 128-token blocks, each block read once per 256 rows instead
// of once per sequence.  Per row every part keeps the running maximum m and sum
// l of an online softmax and the unnormalised output o, and
//   out = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M),   M = max_i m_i,
// over the parts of the prefix and of the row's own tokens.
//
// prefix_kernel.  The (pair of 128-row tiles, KV head, block) units lie on one
// line, cut into equal shares, one per CTA of at most one CTA per SM; a share
// crosses a few segments (pair, KV head) and leaves one partial in each (see
// pkv_prefix_line.h).  Roles hand over through mbarriers, as in the prefill kernel:
//   warps 0-3, 4-7  softmax of stream 0, 1: one row per thread, TMEM lane t;
//   warp 8          issues the MMAs; warp 9 the tensor copies.
// A stream is a row tile with its accumulator.  Two tiles of rows share every
// block (K and V double-buffered); where the second tile of a pair is empty,
// both streams are the first tile, stream t taking every second block in
// buffer t, so the tensor cores still work on one stream under the other's
// softmax.
//   S = Q K^T   tcgen05.mma M 128 x N 128 x K d from shared memory;
//   P           hi + lo 16-bit pairs over S in tensor memory (the weights keep
//               about 16 bits; those of fp16 are off by up to 2^-32 of the row's
//               largest besides: see kRefBelow);
//   O += P V    tcgen05.mma with A from tensor memory, twice per 16 tokens.
// Bound by the softmax and the products taking turns on each stream.  256
// sequences behind 32768 tokens, 32/8 heads of 128: 8192 units in 149 us, 0.92
// PFLOP/s (1.38 with the second product of P); 167 us before the MMAs were issued
// behind elect.sync.  Equal shares replaced a grid of (pair, head, split) with
// the splits picked by a search, which took 299 us for the whole call (227 at
// that step, now 193).  Measured and not kept: steps of 64 tokens with two score
// buffers, as in the biased prefill kernel (193 us for the call against 195: the
// softmax warps' latency bounds both), more registers for the softmax warps by
// setmaxnreg (180, 176 at the time).
//
// own_kernel.  One warp per CTA and per chunk of one sequence's own pages of
// one KV head: the page ring, MMAs and softmax of the single-token decode
// kernel's warp, with nothing to hand over at a segment's end; bound by HBM
// (269 MB of own pages, 256 sequences of up to 512 tokens: 51 us alone and cold,
// 5.5 TB/s of DRAM traffic; the decode kernel's form, which leaves a partial per
// share, took 127).  It depends on nothing the prefix kernel writes and needs little
// of an SM (a 24 KB ring), so its first CTAs start beside the prefix kernel's and
// the rest as SMs come free.  All of it beside the prefix kernel, from a queue, was
// slower: the prefix then took 270 us and the call 301 (227 at the time).
//
// prefix_merge_kernel.  A warp per row adds the parts in a fixed order, four
// warps where rows are few and their parts many; bound by the latency of the
// parts, which are in L2 (17 us alone and cold, about 5 in the same call).
#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_prefix_line.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace px {

constexpr int kRows = kPrefixRows, kTok = kPrefixTok;
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
  static constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;  // TMEM base, abort, max, counts
  static constexpr size_t kSmem = 1024 + kOffMisc + 12 + 4 * kNumBars;
};
template <bool B>
struct Masked {
  static constexpr bool value = B;
};

template <int N>
struct Count {
  static constexpr int value = N;
};
constexpr int64_t kMergeRows = 1024, kMergeParts = 8;

// tokens of the prefix that a sequence of length c sees (bad lengths: none; the
// own kernel reports them)
__device__ __forceinline__ int prefix_len(int c, const PrefixParams& p) {
  return c < 0 || c > p.MBS * kPageSize ? 0 : min(c, p.npb * kPageSize);
}

// What is seen of the prefix, cut over the CTAs that were launched.
__device__ __forceinline__ PrefixLine line_of(const PrefixParams& p, int seen) {
  return PrefixLine(p.Hkv, (int64_t)p.B * (p.Hq / p.Hkv), p.pairs, seen, p.ctas);
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const PrefixParams p, const __grid_constant__ CUtensorMap tmq,
                  const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv) {
  using PL = Plan<D>;
  constexpr int NH = PL::NH;
  constexpr uint32_t kOffK = PL::kOffK, kOffV = PL::kOffV, kOffBar = PL::kOffBar,
                     kOffMisc = PL::kOffMisc;
  const int G = p.Hq / p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * (uint32_t)i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(base_ptr + kOffMisc);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(base_ptr + kOffMisc + 4);
  int32_t* max_len = reinterpret_cast<int32_t*>(base_ptr + kOffMisc + 8);
  volatile int32_t* armed = reinterpret_cast<volatile int32_t*>(base_ptr + kOffMisc + 12);

  if (tid == 0) {
    prefetch_tmap(&tmq);
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
    *abort_flag = 0;
    *max_len = 0;
    for (int i = 0; i < kNumBars; ++i) {
      armed[i] = 0;
      mbar_init(bar(i), (i == kBarPFull || i == kBarPFull + 1) ? kRows / 32 : 1);
    }
    fence_mbar_init();
  }
  __syncthreads();

  // so far nothing of the kernel in front was needed, and it may still run
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the kernel behind this one reads nothing that this one writes before its
  // own end, and everything earlier is complete: it may start
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Tensor memory is taken behind the wait, never before it: a kernel in front
  // that lets this one start may have yet to take its own on the same SM.
  if (warp == 0) {
    tmem_alloc(base + kOffMisc, kTmemCols);
    tmem_relinquish();
  }

  // the positions any sequence sees of the prefix: rows of V behind them may
  // never have been written
  {
    int m = 0;
    for (int b = tid; b < p.B; b += kThreads) m = max(m, prefix_len(p.context_lens[b], p));
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0 && m > 0) atomicMax(max_len, m);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int seen = *max_len;
  const int pages = (seen + kPageSize - 1) / kPageSize;  // those behind are not looked up
  if (blockIdx.x == 0 && tid == 0) *p.seen = seen;  // for the merge
  const PrefixLine line = line_of(p, seen);
  const int64_t lo = blockIdx.x < line.n && seen > 0 ? line.share(blockIdx.x) : 0;
  const int64_t hi = blockIdx.x < line.n && seen > 0 ? line.share(blockIdx.x + 1) : 0;

  // Every role steps through the same parts.  Stream t's i-th block of a part is
  // j0 + i (two tiles) or j0 + 2 i + t (one), in buffer i & 1 or t; use counts
  // of the buffers and the streams run on from part to part (they give the
  // barriers' phases).
  struct Walk {
    PrefixPart s;
    int buf0 = 0, buf1 = 0, str0 = 0, str1 = 0;  // uses before this part
    __device__ int count(int t) const { return s.two ? s.nblk : (s.nblk + 1 - t) / 2; }
    __device__ int block(int t, int i) const { return s.j0 + (s.two ? i : 2 * i + t); }
    __device__ int buf(int t, int i) const { return s.two ? i & 1 : t; }
    __device__ int use(int t, int i) const {
      return (buf(t, i) ? buf1 : buf0) + (s.two ? i >> 1 : i);
    }
    __device__ int str(int t) const { return t ? str1 : str0; }
    __device__ void done() {
      buf0 += (s.nblk + 1) / 2;
      buf1 += s.nblk / 2;
      str0 += count(0);
      str1 += count(1);
    }
  } wk;
  int64_t at = lo;

  auto wait = [&](int i, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(i), parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait_bounded(bar(i), parity, kWaitNs)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp == 9) {
    // ------------------------------------------------------------ copies
    bool ok = true;
    while (ok && next_part(line, at, hi, wk.s)) {
      // Q's tiles are free when every product of the last part with them is done
      for (int bb = 0; ok && bb < 2; ++bb) {
        const int u = bb ? wk.buf1 : wk.buf0;
        if (u > 0)
          ok = __all_sync(0xffffffffu, wait(kBarKFree + bb, (uint32_t)((u - 1) & 1)));
      }
      if (!ok) break;
      if (lane == 0) {
        armed[kBarQ] = armed[kBarQ] + 1;
        const int nq = wk.s.two ? 2 : 1;
        mbar_arrive_expect_tx(bar(kBarQ), (uint32_t)nq * NH * kHalf);
        for (int t = 0; t < nq; ++t)
          for (int c = 0; c < NH; ++c)
            tma_load_3d(base + (uint32_t)(t * NH + c) * kHalf, &tmq, bar(kBarQ), c * 64,
                        wk.s.h * G, (2 * wk.s.pair + t) * (kRows / G));
      }
      const int streams = wk.s.two ? 1 : 2;
      auto entry = [&](int t, int i) -> int {  // lane l < 8: page l's block
        const int pg = wk.block(t, i) * kPages + lane;
        return lane < kPages && t < streams && i < wk.count(t) && pg < pages
                   ? p.prefix_blocks[pg] : 0;
      };
      int cur0 = entry(0, 0), cur1 = entry(1, 0);
      for (int i = 0; ok && i < wk.count(0); ++i) {
        const int nxt0 = entry(0, i + 1), nxt1 = entry(1, i + 1);
        for (int v = 0; ok && v < 2; ++v) {  // K of the streams, then V
          for (int t = 0; t < streams; ++t) {
            if (i >= wk.count(t)) continue;
            const int bb = wk.buf(t, i), u = wk.use(t, i);
            const int npg = min(kPages, pages - wk.block(t, i) * kPages);
            int blk = t == 0 ? cur0 : cur1;
            if (lane < npg && (blk < 0 || blk >= p.NB)) {  // zeros, past the pool
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
              const int r = (blk * p.Hkv + wk.s.h) * kPageSize;
              for (int c = 0; c < NH; ++c)
                tma_load_2d_plain(dst + (uint32_t)c * kHalf,
                                  v ? (const void*)&tmv : (const void*)&tmk, bar(full), c * 64, r);
            }
          }
        }
        ok = ok && !__any_sync(0xffffffffu, *abort_flag != 0);
        cur0 = nxt0;
        cur1 = nxt1;
      }
      wk.done();
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMAs
    if (elect_one()) {
      constexpr uint32_t kIdS = idesc_f16(BF16, false, kRows, kTok);
      constexpr uint32_t kIdO = idesc_f16(BF16, true, kRows, D);
      auto commit = [&](int i) {
        armed[i] = armed[i] + 1;
        umma_commit(bar(i));
      };
      const uint64_t dq = sdesc(base, 16, 1024);
      const uint64_t dk = sdesc(base + kOffK, 16, 1024);
      const uint64_t dv = sdesc(base + kOffV, kHalf, 1024);
      // bb: the buffer; last: nothing uses the buffer after this
      auto qk = [&](int t, int bb, bool two, bool last) {
        const uint64_t a0 = dq + (two && t ? (uint64_t)NH * kHalf >> 4 : 0ull);
        const uint64_t b0 = dk + (bb ? (uint64_t)NH * kHalf >> 4 : 0ull);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (uint32_t)(ks >> 2) * kHalf + (uint32_t)(ks & 3) * 32;
          umma(tmem + (uint32_t)t * kTok, a0 + (off >> 4), b0 + (off >> 4), kIdS, ks > 0);
        }
        commit(kBarSFull + t);
        if (last) commit(kBarKFree + bb);
      };
      // P_t: per 64 tokens 32 columns of hi pairs, then 32 of lo pairs
      auto pv = [&](int t, int bb, bool add, bool last) {
        const uint64_t b0 = dv + (bb ? (uint64_t)NH * kHalf >> 4 : 0ull);
        const uint32_t pt = tmem + (uint32_t)t * kTok;
        const uint32_t dt = tmem + 256 + (uint32_t)t * D;
#pragma unroll
        for (int ks = 0; ks < kTok / 16; ++ks) {
          const uint64_t bv = b0 + ((uint32_t)ks * 16 * 128 >> 4);
          const uint32_t pa = pt + (uint32_t)(ks >> 2) * 64 + (uint32_t)(ks & 3) * 8;
          umma_ts(dt, pa, bv, kIdO, add || ks > 0);
          umma_ts(dt, pa + 32, bv, kIdO, 1);
        }
        commit(kBarODone + t);
        if (last) commit(kBarVFree + bb);
      };
      bool ok = true;
      uint32_t parts = 0;
      // The first product over O_t of a part comes after P_t, which the softmax
      // threads hand over after they have read the last part's O_t out.
      while (ok && next_part(line, at, hi, wk.s)) {
        ok = wait(kBarQ, parts++ & 1);
        if (wk.s.two) {  // one buffer after the other, both streams from it
          const int n = wk.s.nblk;
          uint32_t u0 = (uint32_t)wk.buf0, u1 = (uint32_t)wk.buf1;  // uses of the next block's
          const uint32_t st = (uint32_t)wk.str0, st1 = (uint32_t)wk.str1;
          ok = ok && wait(kBarKFull, u0 & 1);
          if (ok) {
            tc_fence_after();
            qk(0, 0, true, false);
            qk(1, 0, true, true);
          }
          for (int i = 0; ok && i < n; ++i) {
            const int bb = i & 1;
            const bool more = i + 1 < n;
            const uint32_t vu = bb ? u1 : u0, ku = bb ? u0 + 1 : u1;  // this V, the next K
            if (!(ok = wait(kBarPFull, (st + i) & 1) && wait(kBarVFull + bb, vu & 1))) break;
            tc_fence_after();
            pv(0, bb, i > 0, false);
            if (more) {
              if (!(ok = wait(kBarKFull + (bb ^ 1), ku & 1))) break;
              qk(0, bb ^ 1, true, false);
            }
            if (!(ok = wait(kBarPFull + 1, (st1 + i) & 1))) break;
            tc_fence_after();
            pv(1, bb, i > 0, true);
            if (more) qk(1, bb ^ 1, true, true);
            if (bb) {
              ++u0;
              ++u1;
            }
          }
        } else {  // stream t from buffer t
          const int n0 = wk.count(0), n1 = wk.count(1);
          const uint32_t u[2] = {(uint32_t)wk.buf0, (uint32_t)wk.buf1};
          const uint32_t st[2] = {(uint32_t)wk.str0, (uint32_t)wk.str1};
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == 1 && n1 == 0) break;
            ok = ok && wait(kBarKFull + t, u[t] & 1);
            if (!ok) break;
            tc_fence_after();
            qk(t, t, false, true);
          }
          for (int i = 0; ok && i < n0; ++i) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (i >= (t ? n1 : n0)) break;
              ok = wait(kBarPFull + t, (st[t] + i) & 1) && wait(kBarVFull + t, (u[t] + i) & 1);
              if (!ok) break;
              tc_fence_after();
              pv(t, t, i > 0, true);
              if (i + 1 < (t ? n1 : n0)) {
                ok = wait(kBarKFull + t, (u[t] + i + 1) & 1);
                if (!ok) break;
                qk(t, t, false, true);
              }
            }
          }
        }
        wk.done();
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;           // stream
    const int tt = tid - t * kRows;    // row in the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + (uint32_t)t * kTok + lane_base;
    const uint32_t t_o = tmem + 256 + (uint32_t)t * D + lane_base;
    const float c2 = p.scale_log2;
    bool ok = true;
    uint32_t r[32];
    while (ok && next_part(line, at, hi, wk.s)) {
    const int nt = wk.count(t), done = wk.str(t);
    int tok0 = wk.block(t, 0) * kTok;
    const int tok_step = wk.s.two ? kTok : 2 * kTok;
    const int row = (2 * wk.s.pair + (wk.s.two ? t : 0)) * kRows + tt;
    const int b = row / G;
    // last position the row sees; rows past the batch (zero q) see all, unused
    const int vis = (b < p.B ? prefix_len(p.context_lens[b], p) : seen) - 1;
    const int all_vis = __reduce_min_sync(0xffffffffu, vis);
    float m_ref = -INFINITY, l_sum = 0.f;
    for (int i = 0; i < nt; ++i, tok0 += tok_step) {
      // a block outside the pool (reported by the copy warp, zeros in shared
      // memory) is left out: bit pg stands for the step's page pg
      const int pg = tok0 / kPageSize + lane;
      const int entry = lane < kPages && pg < pages ? p.prefix_blocks[pg] : 0;
      ok = __all_sync(0xffffffffu, wait(kBarSFull + t, (uint32_t)((done + i) & 1)));
      if (!ok) break;
      tc_fence_after();
      const uint32_t bad = __ballot_sync(0xffffffffu, entry < 0 || entry >= p.NB);
      const bool full = tok0 + kTok - 1 <= all_vis && bad == 0;
      // last position the row sees in the quarter's pages
      auto vis_of = [&](int qq, int half) { return (bad >> (2 * qq + half)) & 1 ? -1 : vis; };
      uint32_t sa[32], sb[32];
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto qmax = [&](auto mc, const uint32_t (&sq)[32], int qq) {
        const int t0 = tok0 + 32 * qq;
        [[maybe_unused]] const int last[2] = {vis_of(qq, 0), vis_of(qq, 1)};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float a = __uint_as_float(sq[2 * e]), c = __uint_as_float(sq[2 * e + 1]);
          if constexpr (decltype(mc)::value) {
            if (t0 + 2 * e > last[e >> 3]) a = -INFINITY;
            if (t0 + 2 * e + 1 > last[e >> 3]) c = -INFINITY;
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
      const float mx =
          fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c2 - kRefBelow<BF16>;
      const bool grow = mx > m_ref + 8.f;  // lazy rescale, as in the prefill kernel
      float alpha = 1.f;
      if (grow) {
        alpha = ex2(m_ref - mx);
        m_ref = mx;
        l_sum *= alpha;
      }
      if (i > 0) {
        ok = __all_sync(0xffffffffu, wait(kBarODone + t, (uint32_t)((done + i - 1) & 1)));
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
        [[maybe_unused]] const int last[2] = {vis_of(qq, 0), vis_of(qq, 1)};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 y = f2_split(fma2(f2(__uint_as_float(sq[2 * e]),
                                            __uint_as_float(sq[2 * e + 1])), c2x2, nmu2));
          float p0 = ex2(y.x), p1 = ex2(y.y);
          if constexpr (decltype(mc)::value) {
            const int tk = tok0 + 32 * qq + 2 * e;
            if (tk > last[e >> 3]) p0 = 0.f;
            if (tk + 1 > last[e >> 3]) p1 = 0.f;
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
      if (tok0 + kTok > seen && (t == 0 || !wk.s.two)) {
        const int bb = wk.buf(t, i);
        ok = __all_sync(0xffffffffu, wait(kBarVFull + bb, (uint32_t)(wk.use(t, i) & 1)));
        if (!ok) break;
        const int first = max(0, seen - tok0);
        const uint32_t vb = base + kOffV + (uint32_t)bb * NH * kHalf;
        for (int e = tt; e < (kTok - first) * 8 * NH; e += kRows) {
          const int rr = first + e / (8 * NH), ch = e % (8 * NH);
          const uint32_t a = vb + (uint32_t)(ch >> 3) * kHalf + (uint32_t)rr * 128 +
                             (uint32_t)(ch & 7) * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
        }
        // the tensor cores read them through the async proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarPFull + t));
    }
    // ---- the stream's partial: m, l and the unnormalised o of its rows
    if (ok && nt > 0)
      ok = __all_sync(0xffffffffu, wait(kBarODone + t, (uint32_t)((done + nt - 1) & 1)));
    if (!ok) break;
    const int64_t slot = line.slot(blockIdx.x, wk.s.pair, wk.s.h) * 2 + t;
    const bool any = nt > 0 && l_sum != 0.f;  // NaN counts: it has to show
    if (b < p.B) p.pre_ml[slot * kRows + tt] = any ? make_float2(m_ref, l_sum)
                                                   : make_float2(-INFINITY, 0.f);
    if (nt > 0) {
      tc_fence_after();
      float* po = p.pre_o + (slot * kRows + tt) * D;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        tmem_ld32(t_o + (uint32_t)cc * 32, r);
        if (b < p.B) {
#pragma unroll
          for (int e = 0; e < 4; ++e)  // 32 bytes at once: whole sectors
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             po + cc * 32 + 8 * e),
                         "r"(r[8 * e]), "r"(r[8 * e + 1]), "r"(r[8 * e + 2]), "r"(r[8 * e + 3]),
                         "r"(r[8 * e + 4]), "r"(r[8 * e + 5]), "r"(r[8 * e + 6]),
                         "r"(r[8 * e + 7])
                         : "memory");
        }
      }
      tc_fence_before();  // O_t is read before P_t of the next part is handed over
    }
    wk.done();
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

// ---- own parts: 16-bit pages on warp-level MMAs, as in the decode kernel
constexpr int kOwnRing = 3;  // K+V page slots: 24 KB at d 128, what the prefix kernel leaves free
template <int D>
struct OwnPlan {
  static constexpr int kTile = kPageSize * D * 2;  // one K (or V) page
  static constexpr int kStage = 2 * kTile;
  static constexpr size_t kSmem = 1024 + kOwnRing * kStage + 8 * kOwnRing;
};

template <bool BF16, int D, int G>
__global__ void __launch_bounds__(32)
    own_kernel(const PrefixParams p, const __grid_constant__ CUtensorMap tmk,
               const __grid_constant__ CUtensorMap tmv) {
  using PL = OwnPlan<D>;
  constexpr int kMT = D / 16, kBoxes = D * 2 / 128;
  const int lane = threadIdx.x;
  const int chunk = blockIdx.x % p.chunks, seg = blockIdx.x / p.chunks;
  const int b = seg / p.Hkv, h = seg - b * p.Hkv;
  // The kernel before this one reads and writes nothing that matters here, and
  // everything earlier is complete (it waits before it lets this one start).
  // The merge behind waits for this kernel alone, so one CTA ends after both.
  // (The merge may start once every CTA of this kernel has.)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto leave = [&] {
    if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  const int ctx = p.context_lens[b];
  if (ctx < 0 || ctx > p.MBS * kPageSize) {
    if (lane == 0 && chunk == 0 && h == 0) report_error(p.err_word, PKV_ERR_BOUNDS);
    leave();
    return;
  }
  const int np = (ctx + kPageSize - 1) / kPageSize;
  const int first = p.npb + chunk * p.chunk_pages;
  const int n = (chunk == p.chunks - 1 ? np : min(np, first + p.chunk_pages)) - first;
  if (n <= 0) {
    leave();
    return;
  }

  extern __shared__ uint8_t smem_raw[];
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = ring + kOwnRing * PL::kStage;
  if (lane == 0) {
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
    for (int s = 0; s < kOwnRing; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int32_t* table = p.block_tables + (int64_t)b * p.MBS + first;
  // page j's TMA row sits in lane j % 32, 32 pages looked up at a time
  auto look_up = [&](int j0) -> int {
    const int j = j0 + lane;
    if (j >= n) return -1;
    const int blk = table[j];
    if (blk >= 0 && blk < p.NB) return (blk * p.Hkv + h) * kPageSize;
    report_error(p.err_word, PKV_ERR_BOUNDS);
    return -1;
  };
  int cur = look_up(0), nxt = n > 32 ? look_up(32) : -1;  // of pages 32 k .., 32 (k + 1) ..
  int group = 0;
  auto row_of = [&](int j) -> int {  // j / 32 is group or group + 1
    const int a = __shfl_sync(0xffffffffu, cur, j & 31), c = __shfl_sync(0xffffffffu, nxt, j & 31);
    return (j >> 5) == group ? a : c;
  };
  const uint64_t pol = l2_policy_evict_first();
  auto issue = [&](int j) {
    const int row = row_of(j);
    if (lane == 0) {
      const int s = j % kOwnRing;
      const uint32_t kt = ring + (uint32_t)(s * PL::kStage), bar = bars + 8 * s;
      if (row >= 0) {
        mbar_arrive_expect_tx(bar, PL::kStage);
#pragma unroll
        for (int bx = 0; bx < kBoxes; ++bx) {
          tma_load_2d(kt + bx * kPageSize * 128, &tmk, bar, bx * 64, row, pol);
          tma_load_2d(kt + PL::kTile + bx * kPageSize * 128, &tmv, bar, bx * 64, row, pol);
        }
      } else {
        mbar_arrive(bar);
      }
    }
  };
  int issued = 0;
  for (; issued < n && issued < kOwnRing; ++issued) issue(issued);

  // fragment coordinates: see the decode kernel
  const int c4 = lane & 3, r8 = lane >> 2;
  const int qk_tok = (lane & 7) + ((lane >> 3) & 1) * 8, qk_hi = lane >> 4;
  const int pv_tok = (lane & 7) + (lane >> 4) * 8, pv_hi = (lane >> 3) & 1;
  auto swz = [](int tok, int chunk16) -> uint32_t {
    return (uint32_t)((chunk16 >> 3) * (kPageSize * 128) + tok * 128 +
                      (((chunk16 & 7) ^ (tok & 7)) << 4));
  };
  uint32_t qf[kMT][2];
  {
    const bool real = r8 < G;
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(
        static_cast<const uint16_t*>(p.q) + ((int64_t)b * p.Hq + h * G + (real ? r8 : 0)) * D);
#pragma unroll
    for (int ks = 0; ks < kMT; ++ks) {
      qf[ks][0] = real ? qrow[8 * ks + c4] : 0;
      qf[ks][1] = real ? qrow[8 * ks + c4 + 4] : 0;
    }
  }
  float o[kMT][4], m2[2] = {-INFINITY, -INFINITY}, l2[2] = {0.f, 0.f};
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[mt][e] = 0.f;
  const float c2 = p.scale_log2;

  auto pages = [&](auto npc, const uint32_t* kt, const int* rem) {
    constexpr int NP = decltype(npc)::value;
    float x[NP][4];
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < kMT; ++ks) {
        uint32_t a[4];
        ldsm_x4(a, kt[i] + swz(qk_tok, 2 * ks + qk_hi));
        if (ks & 1) mma_16816<BF16>(s1, a, qf[ks][0], qf[ks][1]);
        else mma_16816<BF16>(s0, a, qf[ks][0], qf[ks][1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = (s0[e] + s1[e]) * c2;
      if (rem[i] < kPageSize) {
        if (r8 >= rem[i]) x[i][0] = x[i][1] = -INFINITY;
        if (r8 + 8 >= rem[i]) x[i][2] = x[i][3] = -INFINITY;
      }
      mx0 = fmaxf(mx0, fmaxf(x[i][0], x[i][2]));
      mx1 = fmaxf(mx1, fmaxf(x[i][1], x[i][3]));
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
    }
    constexpr float kBelow = kRefBelow<BF16>, kGrowth = 8.f + kBelow;
    if (__any_sync(0xffffffffu, mx0 > m2[0] + kGrowth || mx1 > m2[1] + kGrowth)) {  // lazy rescale
      const float n0 = fmaxf(m2[0], mx0 - kBelow), n1 = fmaxf(m2[1], mx1 - kBelow);
      const float a0 = n0 == -INFINITY ? 1.f : ex2(m2[0] - n0);
      const float a1 = n1 == -INFINITY ? 1.f : ex2(m2[1] - n1);
      m2[0] = n0;
      m2[1] = n1;
      l2[0] *= a0;
      l2[1] *= a1;
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        o[mt][0] *= a0;
        o[mt][1] *= a1;
        o[mt][2] *= a0;
        o[mt][3] *= a1;
      }
    }
    const float mu0 = m2[0] == -INFINITY ? 0.f : m2[0], mu1 = m2[1] == -INFINITY ? 0.f : m2[1];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float p0 = ex2(x[i][0] - mu0), p1 = ex2(x[i][1] - mu1);
      const float p2 = ex2(x[i][2] - mu0), p3 = ex2(x[i][3] - mu1);
      l2[0] += p0 + p2;
      l2[1] += p1 + p3;
      const uint32_t h01 = pack2<BF16>(p0, p1), h23 = pack2<BF16>(p2, p3);
      const float2 f01 = unpack2<BF16>(h01), f23 = unpack2<BF16>(h23);
      const uint32_t l01 = pack2<BF16>(p0 - f01.x, p1 - f01.y);
      const uint32_t l23 = pack2<BF16>(p2 - f23.x, p3 - f23.y);
      const uint32_t vt = kt[i] + PL::kTile;
      if (rem[i] < kPageSize) {  // rows of V past the end may hold anything (0 x NaN)
        const int nz = (kPageSize - rem[i]) * kBoxes * 8;
        for (int e = lane; e < nz; e += 32) {
          const int rr = rem[i] + e / (kBoxes * 8), bx = (e / 8) % kBoxes;
          const uint32_t a = vt + (uint32_t)(bx * kPageSize * 128 + rr * 128 + (e % 8) * 16);
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      const uint32_t bh0 = movm_trans(h01), bh1 = movm_trans(h23);
      const uint32_t bl0 = movm_trans(l01), bl1 = movm_trans(l23);
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        uint32_t a[4];
        ldsm_x4_trans(a, vt + swz(pv_tok, 2 * mt + pv_hi));
        mma_16816<BF16>(o[mt], a, bh0, bh1);
        mma_16816<BF16>(o[mt], a, bl0, bl1);
      }
    }
  };
  auto ready = [&](int j) -> bool {
    return mbar_wait_bounded(bars + 8 * (j % kOwnRing), (uint32_t)((j / kOwnRing) & 1), kWaitNs);
  };
  bool ok = true;
  for (int j = 0; j < n;) {
    const int k = n - j >= 2 ? 2 : 1;
    uint32_t kt[2];
    int rem[2];
    bool valid = true;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i < k) {
        ok = ok && __all_sync(0xffffffffu, ready(j + i));
        kt[i] = ring + (uint32_t)((j + i) % kOwnRing) * PL::kStage;
        rem[i] = min(kPageSize, ctx - (first + j + i) * kPageSize);
        if (row_of(j + i) < 0) valid = false;
      }
    }
    if (!ok) break;
    if (k == 2 && valid) {
      pages(Count<2>{}, kt, rem);
    } else {
      for (int i = 0; i < k; ++i)
        if (row_of(j + i) >= 0) pages(Count<1>{}, kt + i, rem + i);
    }
    __syncwarp();
    j += k;
    // the look-up of the group after the one in nxt starts when j enters nxt
    if ((j >> 5) != group && j < n) {
      group = j >> 5;
      cur = nxt;
      nxt = (group + 1) * 32 < n ? look_up((group + 1) * 32) : -1;
    }
    for (; issued < n && issued < j + kOwnRing; ++issued) issue(issued);
  }
  if (!ok) {  // a copy never came: let those in flight land, then report
    if (lane == 0) report_error(p.err_word, PKV_ERR_TIMEOUT);
    for (int s = 0; s < kOwnRing; ++s) {
      const int last = issued - 1 - s;
      if (last >= 0) ready(last);
    }
    leave();
    return;
  }

#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l2[0] += __shfl_xor_sync(0xffffffffu, l2[0], off);
    l2[1] += __shfl_xor_sync(0xffffffffu, l2[1], off);
  }
  const int64_t slot = (int64_t)seg * p.chunks + chunk;
  const int h0 = 2 * c4, h1 = h0 + 1;
  if (r8 == 0) {
    if (h0 < G) p.own_ml[slot * G + h0] = make_float2(m2[0], l2[0]);
    if (h1 < G) p.own_ml[slot * G + h1] = make_float2(m2[1], l2[1]);
  }
  float* po = p.own_o + slot * G * D;
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt) {
    const int dA = 16 * mt + r8;
    if (h0 < G) {
      po[h0 * D + dA] = o[mt][0];
      po[h0 * D + dA + 8] = o[mt][2];
    }
    if (h1 < G) {
      po[h1 * D + dA] = o[mt][1];
      po[h1 * D + dA + 8] = o[mt][3];
    }
  }
  leave();
}

// ---- the merge: WPR warps per row, kMergeWarps warps per CTA.  A warp's lanes
// hold the row's d columns and take every WPR-th part, 4 loads in flight.
constexpr int kMergeWarps = 4;
template <int D, int WPR>
__global__ void __launch_bounds__(kMergeWarps * 32) prefix_merge_kernel(const PrefixParams p) {
  constexpr int V = D / 32;  // columns per lane
  // a kernel behind this one that waits for its end may start its prologue
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
  const int64_t orow = (int64_t)blockIdx.x * (kMergeWarps / WPR) + warp / WPR;  // b Hq + hq
  const bool real = orow < (int64_t)p.B * p.Hq;
  float acc[V], l = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  if (real) {
    const int b = (int)(orow / p.Hq), hq = (int)(orow - (int64_t)b * p.Hq);
    const int G = p.Hq / p.Hkv, h = hq / G, gi = hq - h * G;
    // the row's parts: stream by stream of the prefix, then its own chunks
    const int row = b * G + gi, tile = row >> 7, pair = tile >> 1, rr = row & 127;
    const int seen = *p.seen;
    int npre = 0, streams = 1;
    int64_t pre0 = 0;
    if (seen > 0) {
      const PrefixLine line = line_of(p, seen);
      const bool two = line.weight(pair) == 2;
      const int64_t c0 = line.first_cta(pair, h), c1 = line.last_cta(pair, h);
      streams = two ? 1 : 2;
      npre = (int)(c1 - c0 + 1) * streams;
      pre0 = line.slot(c0, pair, h) * 2 + (two ? tile & 1 : 0);
    }
    const int ctx = p.context_lens[b];
    const int own = ctx < 0 || ctx > p.MBS * kPageSize
                        ? 0 : max(0, (ctx + kPageSize - 1) / kPageSize - p.npb);
    const int nown = min(p.chunks, (own + p.chunk_pages - 1) / p.chunk_pages);
    const int64_t own0 = ((int64_t)(b * p.Hkv + h) * p.chunks) * G + gi;
    const int n = npre + nown;
    auto ml_of = [&](int k) -> float2 {
      return k < npre ? p.pre_ml[(pre0 + (streams == 2 ? k : 2 * k)) * kRows + rr]
                      : p.own_ml[own0 + (int64_t)(k - npre) * G];
    };
    auto o_of = [&](int k) -> const float* {
      return (k < npre ? p.pre_o + ((pre0 + (streams == 2 ? k : 2 * k)) * kRows + rr) * D
                       : p.own_o + (own0 + (int64_t)(k - npre) * G) * D) + lane * V;
    };
    float2 mine = make_float2(-INFINITY, 0.f);  // part `lane`
    if (lane < n) mine = ml_of(lane);
    float M = mine.x;
    for (int k = lane + 32; k < n; k += 32) M = fmaxf(M, ml_of(k).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.f;  // nothing at all, or nothing but NaN
    for (int k0 = 0; k0 < n; k0 += 32) {
      if (k0 > 0) mine = k0 + lane < n ? ml_of(k0 + lane) : make_float2(-INFINITY, 0.f);
      const float wl = ex2(mine.x - M);
      const int m = min(32, n - k0);
#pragma unroll 8
      for (int k = sub; k < m; k += WPR) {
        const float w = __shfl_sync(0xffffffffu, wl, k), ll = __shfl_sync(0xffffffffu, mine.y, k);
        if (ll != 0.f) {  // a part with nothing in it was not written
          l += w * ll;
          const float* x = o_of(k0 + k);
          if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4*>(x);
            acc[0] += w * v.x;
            acc[1] += w * v.y;
            acc[2] += w * v.z;
            acc[3] += w * v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(x);
            acc[0] += w * v.x;
            acc[1] += w * v.y;
          }
        }
      }
    }
  }
  if constexpr (WPR > 1) {
    __shared__ float sh[kMergeWarps][D + 1];
#pragma unroll
    for (int e = 0; e < V; ++e) sh[warp][lane * V + e] = acc[e];
    if (lane == 0) sh[warp][D] = l;
    __syncthreads();
    if (sub != 0) return;
    for (int w = 1; w < WPR; ++w) {
      l += sh[warp + w][D];
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += sh[warp + w][lane * V + e];
    }
  }
  if (!real) return;
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] *= inv;
  const int64_t at = orow * D + lane * V;
  if (p.out_dtype == PKV_F32) {
#pragma unroll
    for (int e = 0; e < V; ++e) static_cast<float*>(p.out)[at + e] = acc[e];
  } else {
    const bool bf = p.out_dtype == PKV_BF16;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at);
#pragma unroll
    for (int e = 0; e < V / 2; ++e)
      out[e] = bf ? pack2<true>(acc[2 * e], acc[2 * e + 1])
                  : pack2<false>(acc[2 * e], acc[2 * e + 1]);
  }
}

// Every kernel may start before the one in front of it has ended (see the waits).
template <typename... KP, typename... A>
cudaError_t launch_behind(void (*kern)(KP...), unsigned grid, unsigned block, size_t smem,
                          cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool BF16, int D>
cudaError_t launch(const PrefixLaunch& l) {
  const int G = l.p.Hq / l.p.Hkv;
  auto pre = prefix_kernel<BF16, D>;
  auto own = G == 1 ? own_kernel<BF16, D, 1> : G == 2 ? own_kernel<BF16, D, 2>
             : G == 4 ? own_kernel<BF16, D, 4> : own_kernel<BF16, D, 8>;
  static std::atomic<uint64_t> configured{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(pre, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Plan<D>::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  static_assert(OwnPlan<D>::kSmem <= 48 * 1024, "no attribute needed");
  e = launch_behind(pre, (unsigned)l.p.ctas, kThreads, Plan<D>::kSmem, l.stream, l.p, l.tmap_q,
                    l.tmap_k, l.tmap_v);
  if (e != cudaSuccess) return e;
  e = launch_behind(own, (unsigned)((int64_t)l.p.B * l.p.Hkv * l.p.chunks), 32, OwnPlan<D>::kSmem,
                    l.stream, l.p, l.tmap_k, l.tmap_v);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)l.p.B * l.p.Hq;
  // a warp per row where rows are many and their parts few
  const int64_t segs = (int64_t)l.p.pairs * l.p.Hkv;
  if (rows >= kMergeRows && l.sms < kMergeParts * segs)
    return launch_behind(prefix_merge_kernel<D, 1>,
                         (unsigned)((rows + kMergeWarps - 1) / kMergeWarps), kMergeWarps * 32, 0,
                         l.stream, l.p);
  return launch_behind(prefix_merge_kernel<D, kMergeWarps>, (unsigned)rows, kMergeWarps * 32, 0,
                       l.stream, l.p);
}

}  // namespace px

cudaError_t launch_prefix(const PrefixLaunch& l) {
  if (l.d == 64) return l.bf16 ? px::launch<true, 64>(l) : px::launch<false, 64>(l);
  if (l.d == 128) return l.bf16 ? px::launch<true, 128>(l) : px::launch<false, 128>(l);
  return cudaErrorNotSupported;
}

}  // namespace pkv
