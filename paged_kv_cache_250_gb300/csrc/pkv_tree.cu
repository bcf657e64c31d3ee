// Decode attention for trees of drafted tokens, on the 5th-generation tensor
// cores.
//
// The n nodes of a sequence's tree times the g query heads of a KV head are the
// rows of a dense product with the sequence's cached blocks: every row sees the
// whole past, and of the tree's own positions those its 64-bit mask names.  Per
// row every part keeps the running maximum m and sum l of an online softmax and
// the unnormalised output o, and
//   out = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M),   M = max_i m_i.
//
// tree_kernel.  Persistent, at most one CTA per SM; the segments (sequence, KV
// head, rows) lie on two lines of costs, cut into equal shares (see
// pkv_tree_line.h), so that ragged contexts and one long one both fill the GPU.
// A segment wholly inside a share is normalised and written at once; one that is
// cut leaves a partial in each share: slot 2 c where it came from the share
// before, 2 c + 1 where it starts in share c.  Roles hand over through mbarriers:
//   warps 0-7, 8-15 softmax of stream 0, 1: a row is two threads';
//   warps 16, 17    the tensor copies; warps 18, 19 issue the MMAs.
// A stream is a row tile with its accumulator.
//   Line 2, segments of two tiles: a share per CTA.  Both streams take every
//   block, K and V double-buffered and copied by a warp each; one warp issues.
//   Line 1, segments of one tile (up to 128 rows: the usual tree), after it: a
//   share per stream, with a K and a V buffer, a copying and an issuing warp of
//   its own, so that one stream's segment ends, copies and products run under the
//   other's softmax.
//   S = Q K^T   tcgen05.mma M 128 x N 128 x K d from shared memory;
//   P           hi + lo 16-bit pairs over S in tensor memory (the weights keep
//               about 16 bits; those of fp16 are off by up to 2^-32 of the row's
//               largest besides: see kRefBelow);
//   O += P V    tcgen05.mma with A from tensor memory, twice per 16 tokens.
// One tile is bound by HBM: 8 x 32768 tokens of 8 KV heads and 8 nodes, 1.07 GB, 180
// us, 6.0 TB/s (235 us while one warp copied K and V of both streams in turn: it
// waited for one stream's buffer while the other's was free).  Two tiles are bound by
// each stream's chain of softmax (2200 cycles per block) and products (2200): 263 us
// for the same cache and 64 nodes, 1.0 PFLOP/s counted, 1.6 with the second product
// of P; the tensor pipe is active 73 % of the cycles.  Short segments and small calls
// are bound by latency: 64 sequences of 512 tokens 42 us, of 128 tokens 20, one of 708
// tokens 10.7, of which 3 are the merge behind.  A launch fetches its code anew, so
// short code counts: scores masked in tensor memory before the softmax, instead of a
// second softmax with masks, and one copy of it for both lines took a cold launch of
// the smallest call from 24 to 15 us.
// Measured and not kept: both streams on one segment with a join at its end (tree of
// 32 ragged sequences 120 us, now 83); K and V prefetched into L2 by the copy warp
// (176 -> 290 us: its look-ups held up its copies); P handed over in two halves (280
// -> 277, ragged trees 97 -> 102); 32 scores at a time (280 -> 289); a quarter of the
// powers of two as a polynomial on the FMA pipe (280 -> 296).
//
// tree_merge_kernel joins the parts of the cut segments, in order.
#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"
#include "pkv_tree_line.h"

namespace pkv {
namespace tr {

constexpr int kRows = kTreeRows, kTok = kTreeTok;
constexpr int kPages = kTok / kPageSize;
constexpr int kThreads = 640, kSoft = 256;  // of them for each stream's softmax
constexpr uint32_t kHalf = 16384;  // 128 rows x 128 bytes: 64 d columns of a tile or block
// one barrier per buffer or stream, in pairs
constexpr int kBarQ = 0, kBarQFree = 2, kBarKFull = 4, kBarVFull = 6, kBarKFree = 8,
              kBarVFree = 10, kBarSFull = 12, kBarPFull = 14, kBarODone = 16, kNumBars = 18;
constexpr uint32_t kTmemCols = 512;  // S0/P0, S1/P1, then O0, O1
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kWarpCopy = 2 * kSoft / 32, kWarpMma = kWarpCopy + 2;  // two each
constexpr int kSeqs = 128;  // sequences whose rows and lengths are at hand in shared memory

template <int D>
struct Plan {
  static constexpr int NH = D / 64;
  static constexpr uint32_t kOffK = 2 * NH * kHalf;
  static constexpr uint32_t kOffV = 4 * NH * kHalf;
  static constexpr uint32_t kOffX = 6 * NH * kHalf;             // [2][2][2][128]: see softmax
  static constexpr uint32_t kOffBar = kOffX + 4 * 8 * kRows;
  static constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;     // TMEM base, abort, counts
  static constexpr uint32_t kOffSeq = (kOffMisc + 24 + 4 * kNumBars + 15) / 16 * 16;  // [kSeqs]
  static constexpr uint32_t kOffBounds = kOffSeq + 16 * kSeqs;  // [3]
  static constexpr uint32_t kOffPfx = kOffBounds + 48;          // [2][B+1]
  static constexpr size_t smem(int B) { return 1024 + kOffPfx + 8 * ((size_t)B + 1); }
};
static_assert(Plan<128>::smem(kTreeMaxBatch) <= 227 * 1024, "the largest batch fits");

// Rows and length of sequence b; none where they break the rules.
__device__ __forceinline__ bool seq_of(const TreeParams& p, int b, int& q0, int& n, int& ctx) {
  q0 = p.q_start[b];
  const int q1 = p.q_start[b + 1];
  ctx = p.context_lens[b];
  n = q1 - q0;
  if (q0 >= 0 && q1 >= q0 && n <= p.max_q && q1 <= p.total_q && ctx >= n &&
      ctx <= p.MBS * kPageSize)
    return true;
  n = 0;
  return false;
}

// 32 bytes at once: a whole sector
__device__ __forceinline__ void store32(void* to, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// a 16-bit pair in fp32; bf16 in an instruction each (the conversion functions took
// 59 more per warp and block: 274 us for 8 x 32768 tokens and 64 nodes, now 266)
template <bool BF16>
__device__ __forceinline__ float2 floats_of(uint32_t u) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  else
    return unpack2<false>(u);
}

// Partial rows lie in groups of 32, eight columns of each row after the other: what a
// warp stores at once (a piece of each lane's row) is contiguous, where rows of their
// own took a line per lane (64 nodes behind 701 tokens 17.5 us, now 16.4).  A row's
// first piece, and the steps to the next:
template <int D>
__device__ __forceinline__ int64_t part_at(int64_t row) {
  return (row & ~31ll) * D + (row & 31) * 8;
}
constexpr int kPartStep = 32 * 8;

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tmq,
                const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv) {
  using PL = Plan<D>;
  constexpr int NH = PL::NH;
  constexpr uint32_t kOffK = PL::kOffK, kOffV = PL::kOffV;
  const int G = p.Hq / p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  auto bar = [&](int i) -> uint32_t { return base + PL::kOffBar + 8u * (uint32_t)i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(base_ptr + PL::kOffMisc);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(base_ptr + PL::kOffMisc + 4);
  volatile int32_t* armed = reinterpret_cast<volatile int32_t*>(base_ptr + PL::kOffMisc + 8);
  volatile uint32_t* bad_pages = reinterpret_cast<volatile uint32_t*>(
      base_ptr + PL::kOffMisc + 8 + 4 * kNumBars);  // of K's buffers, two uses each
  int4* seqs = reinterpret_cast<int4*>(base_ptr + PL::kOffSeq);  // (q0, n, ctx)
  uint4* bounds = reinterpret_cast<uint4*>(base_ptr + PL::kOffBounds);
  uint32_t* pfx = reinterpret_cast<uint32_t*>(base_ptr + PL::kOffPfx);  // [2][B+1] costs before

  if (tid == 0) {
    prefetch_tmap(&tmq);
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
    *abort_flag = 0;
    for (int i = 0; i < kNumBars; ++i) {
      armed[i] = 0;
      mbar_init(bar(i), (i == kBarPFull || i == kBarPFull + 1) ? kSoft / 32 : 1);
    }
    fence_mbar_init();
    pfx[0] = 0;
    pfx[p.B + 1] = 0;
  }
  // so far nothing of the kernel in front was needed, and it may still run
  griddep_wait_then_trigger();
  // Tensor memory is taken behind the wait, never before it: a kernel in front
  // that lets this one start may have yet to take its own on the same SM.
  if (warp == 0) {
    tmem_alloc(base + PL::kOffMisc, kTmemCols);
    tmem_relinquish();
  }
  for (int b = tid; b < p.B; b += kThreads) {
    int q0, n, ctx;
    if (!seq_of(p, b, q0, n, ctx) && blockIdx.x == 0) report_error(p.err_word, PKV_ERR_BOUNDS);
    if (b < kSeqs) seqs[b] = make_int4(q0, n, ctx, 0);
    const int nblk = tree_blocks(ctx);
    pfx[b + 1] = (uint32_t)tree_seq_cost(false, p.Hkv, n * G, nblk);
    pfx[p.B + 1 + b + 1] = (uint32_t)tree_seq_cost(true, p.Hkv, n * G, nblk);
  }
  __syncthreads();
  if (warp < 2) {  // inclusive scans, a warp per line
    uint32_t* line = pfx + warp * (p.B + 1);
    uint32_t carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int i = b0 + lane + 1;
      uint32_t v = i <= p.B ? line[i] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += u;
      }
      if (i <= p.B) line[i] = v + carry;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Every role steps through the parts of a share.
  struct Walk {
    TreePart s;
    int q0, n, ctx;      // first row of q, nodes, length
    uint32_t at, hi;     // costs
    int share;
  } wk;
  const uint32_t* line = pfx;
  bool two = false;
  // k: the CTA's share of line 2 (0), its streams' of line 1 (1, 2), whose first
  // shares go to CTAs of their own.  Their bounds are looked up once, by a thread each.
  const int grid = gridDim.x;
  if (tid < 3) {
    const uint32_t* ln = pfx + (tid == 0 ? p.B + 1 : 0);
    const int share = tid < 2 ? blockIdx.x : grid + blockIdx.x;
    const int64_t cost = ln[p.B], n = tree_shares(cost, tid == 0 ? grid : 2 * grid);
    uint32_t from = 0, to = 0;
    int a = 0;  // the sequence holding `from`: the last with ln <= from
    if (share < n && cost > 0) {
      from = (uint32_t)tree_share(share, cost, n);
      to = (uint32_t)tree_share(share + 1, cost, n);
      for (int z = p.B; z - a > 1;) {
        const int mid = (a + z) >> 1;
        if (ln[mid] <= from) a = mid; else z = mid;
      }
    }
    bounds[tid] = make_uint4(from, to, (uint32_t)a, (uint32_t)share);
  }
  __syncthreads();
  auto begin = [&](int k) {
    const uint4 v = bounds[k];
    two = k == 0;
    line = pfx + (two ? p.B + 1 : 0);
    wk.at = v.x;
    wk.hi = v.y;
    wk.s.b = (int)v.z;
    wk.share = (int)v.w;
  };
  auto next = [&]() -> bool {
    while (wk.at < wk.hi) {
      while (line[wk.s.b + 1] <= wk.at) ++wk.s.b;
      if (wk.s.b < kSeqs) {
        const int4 v = seqs[wk.s.b];
        wk.q0 = v.x;
        wk.n = v.y;
        wk.ctx = v.z;
      } else {
        seq_of(p, wk.s.b, wk.q0, wk.n, wk.ctx);
      }
      wk.at += tree_part(two, wk.n * G, tree_blocks(wk.ctx), wk.at - line[wk.s.b], wk.hi - wk.at,
                         wk.s);
      if (wk.s.nblk > 0) return true;
    }
    return false;
  };
  auto wait = [&](int i, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(i), parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait_bounded(bar(i), parity, kWaitNs)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp == kWarpCopy || warp == kWarpCopy + 1) {
    // ------------------------------------------------------------ copies
    bool ok = true;
    // uses of the buffers and Q slots so far: they give the barriers' phases
    int ku[2] = {0, 0}, vu[2] = {0, 0}, qu[2] = {0, 0};
    auto load_q = [&](int sl, int row) {
      if (qu[sl] > 0)
        ok = __all_sync(0xffffffffu, wait(kBarQFree + sl, (uint32_t)((qu[sl] - 1) & 1)));
      ++qu[sl];
      if (!ok || lane != 0) return;
      armed[kBarQ + sl] = armed[kBarQ + sl] + 1;
      mbar_arrive_expect_tx(bar(kBarQ + sl), NH * kHalf);
      for (int c = 0; c < NH; ++c)
        tma_load_3d(base + (uint32_t)(sl * NH + c) * kHalf, &tmq, bar(kBarQ + sl), c * 64,
                    wk.s.h * G, wk.q0 + row / G);
    };
    // block j (table entries in lanes 0 to 7) of V or K into buffer bb, used u times
    auto load = [&](bool v, int bb, int u, int j, int blk) {
      const int npg = min(kPages, (wk.ctx + kPageSize - 1) / kPageSize - j * kPages);
      const bool gone = lane < npg && (blk < 0 || blk >= p.NB);
      if (gone) {  // zeros, past the pool
        if (!v) report_error(p.err_word, PKV_ERR_BOUNDS);
        blk = p.NB;
      }
      const uint32_t bad = __ballot_sync(0xffffffffu, gone);
      const int full = (v ? kBarVFull : kBarKFull) + bb;
      if (u > 0)
        ok = __all_sync(0xffffffffu,
                        wait((v ? kBarVFree : kBarKFree) + bb, (uint32_t)((u - 1) & 1)));
      if (!ok) return;
      if (lane == 0) {
        armed[full] = armed[full] + 1;
        if (!v) bad_pages[2 * bb + (u & 1)] = bad;  // read behind the product with this K
        mbar_arrive_expect_tx(bar(full), (uint32_t)npg * NH * kPageSize * 128);
      }
      __syncwarp();
      if (lane < npg) {
        const uint32_t dst = base + (v ? kOffV : kOffK) + (uint32_t)bb * NH * kHalf +
                             (uint32_t)lane * kPageSize * 128;
        const int r = (blk * p.Hkv + wk.s.h) * kPageSize;
        for (int c = 0; c < NH; ++c)
          tma_load_2d_plain(dst + (uint32_t)c * kHalf, v ? (const void*)&tmv : (const void*)&tmk,
                            bar(full), c * 64, r);
      }
    };
    auto entry = [&](int j) -> int {  // lane l < 8: the block of page l of block j
      const int pg = j * kPages + lane;
      return lane < kPages && j < wk.s.j0 + wk.s.nblk && pg < (wk.ctx + kPageSize - 1) / kPageSize
                 ? p.block_tables[(int64_t)wk.s.b * p.MBS + pg] : 0;
    };
    const bool v = warp != kWarpCopy;
    begin(0);  // the first warp: Q and K, the second: V
    while (ok && next()) {
      int cur = entry(wk.s.j0);
      for (int t = 0; ok && t < 2; ++t) {
        if (v) ++qu[t];
        else load_q(t, wk.s.row0 + t * kRows);
      }
      for (int i = 0; ok && i < wk.s.nblk; ++i) {
        const int nxt = entry(wk.s.j0 + i + 1);
        load(v, i & 1, v ? vu[i & 1] : ku[i & 1], wk.s.j0 + i, cur);
        ++ku[i & 1];
        ++vu[i & 1];
        cur = nxt;
      }
    }
    // The second warp goes on to stream 1's line when the first has issued all of line
    // 2: it never waited for Q's slots, and phases are told apart by parity only while
    // at most one is outstanding.
    __syncwarp();
    asm volatile("bar.sync 10, 64;" ::: "memory");
    const int t = warp - kWarpCopy;
    begin(1 + t);  // each a stream
    while (ok && next()) {
      int cur = entry(wk.s.j0);
      load_q(t, wk.s.row0);
      for (int i = 0; ok && i < wk.s.nblk; ++i) {
        const int nxt = entry(wk.s.j0 + i + 1);
        load(false, t, t ? ku[1]++ : ku[0]++, wk.s.j0 + i, cur);
        if (ok) load(true, t, t ? vu[1]++ : vu[0]++, wk.s.j0 + i, cur);
        cur = nxt;
      }
    }
  } else if (warp >= kWarpMma) {
    // ------------------------------------------------------------ MMAs
    // blocks of each stream and uses of each buffer so far, segments so far
    uint32_t st = 0, u0 = 0, u1 = 0, segs = 0;
    bool ok = true;
    constexpr uint32_t kIdS = idesc_f16(BF16, false, kRows, kTok);
    constexpr uint32_t kIdO = idesc_f16(BF16, true, kRows, D);
    auto commit = [&](int i) {
      armed[i] = armed[i] + 1;
      umma_commit(bar(i));
    };
    const uint64_t dq = sdesc(base, 16, 1024);
    const uint64_t dk = sdesc(base + kOffK, 16, 1024);
    const uint64_t dv = sdesc(base + kOffV, kHalf, 1024);
    // Q's slot t; bb: the buffer; last: nothing uses the buffer after this; q_last:
    // nothing uses the slot
    auto qk = [&](int t, int bb, bool last, bool q_last) {
      const uint64_t a0 = dq + (t ? (uint64_t)NH * kHalf >> 4 : 0ull);
      const uint64_t b0 = dk + (bb ? (uint64_t)NH * kHalf >> 4 : 0ull);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = (uint32_t)(ks >> 2) * kHalf + (uint32_t)(ks & 3) * 32;
        umma(tmem + (uint32_t)t * kTok, a0 + (off >> 4), b0 + (off >> 4), kIdS, ks > 0);
      }
      commit(kBarSFull + t);
      if (last) commit(kBarKFree + bb);
      if (q_last) commit(kBarQFree + t);
    };
    // P_t: per 16 tokens eight columns of hi pairs, then eight of lo pairs
    auto pv = [&](int t, int bb, bool add, bool last) {
      const uint64_t b0 = dv + (bb ? (uint64_t)NH * kHalf >> 4 : 0ull);
      const uint32_t pt = tmem + (uint32_t)t * kTok;
      const uint32_t dt = tmem + 256 + (uint32_t)t * D;
#pragma unroll
      for (int ks = 0; ks < kTok / 16; ++ks) {
        const uint64_t bv = b0 + ((uint32_t)ks * 16 * 128 >> 4);
        umma_ts(dt, pt + (uint32_t)ks * 16, bv, kIdO, add || ks > 0);
        umma_ts(dt, pt + (uint32_t)ks * 16 + 8, bv, kIdO, 1);
      }
      commit(kBarODone + t);
      if (last) commit(kBarVFree + bb);
    };
    // The first product over O_t of a part comes after P_t, which the softmax
    // threads hand over after they have read the last part's O_t out.
    if (elect_one()) {
      begin(0);
      while (ok && next()) {  // one buffer after the other, both streams from it
        const int n = wk.s.nblk;
        if (warp == kWarpMma) {  // (the other counts)
          uint32_t a0 = u0, a1 = u1;  // uses of the next block's buffer
          ok = wait(kBarKFull, a0 & 1) && wait(kBarQ, segs & 1) && wait(kBarQ + 1, segs & 1);
          if (!ok) break;
          tc_fence_after();
          qk(0, 0, false, n == 1);
          qk(1, 0, true, n == 1);
          for (int i = 0; ok && i < n; ++i) {
            const int bb = i & 1;
            const bool more = i + 1 < n, end = i + 2 == n;
            const uint32_t vu = bb ? a1 : a0, ku = bb ? a0 + 1 : a1;  // this V, the next K
            if (!(ok = wait(kBarPFull, (st + i) & 1) && wait(kBarVFull + bb, vu & 1))) break;
            tc_fence_after();
            pv(0, bb, i > 0, false);
            if (more) {
              if (!(ok = wait(kBarKFull + (bb ^ 1), ku & 1))) break;
              qk(0, bb ^ 1, false, end);
            }
            if (!(ok = wait(kBarPFull + 1, (st + i) & 1))) break;
            tc_fence_after();
            pv(1, bb, i > 0, true);
            if (more) qk(1, bb ^ 1, true, end);
            if (bb) {
              ++a0;
              ++a1;
            }
          }
        }
        u0 += (n + 1) / 2;
        u1 += n / 2;
        st += n;
        ++segs;
      }
    }
    // Then a stream each, whose products are a chain.  The second warp begins when the
    // first has issued all of line 2 (no earlier: a barrier's phases are told apart by
    // parity) and stream 1's last product of it, which is another thread's, is done.
    __syncwarp();
    asm volatile("bar.sync 1, 64;" ::: "memory");
    if (elect_one()) {  // the lane that was elected before
      const int t = warp != kWarpMma;
      uint32_t u = t ? u1 : u0;
      if (t == 1 && st > 0) {
        ok = wait(kBarODone + 1, (st - 1) & 1);
        tc_fence_after();
      }
      begin(1 + t);
      while (ok && next()) {
        ok = wait(kBarQ + t, segs++ & 1);
        for (int i = 0; ok && i < wk.s.nblk; ++i, ++u, ++st) {
          if (!(ok = wait(kBarKFull + t, u & 1))) break;
          tc_fence_after();
          qk(t, t, true, i + 1 == wk.s.nblk);
          if (!(ok = wait(kBarPFull + t, st & 1) && wait(kBarVFull + t, u & 1))) break;
          tc_fence_after();
          pv(t, t, i > 0, true);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    // A row is two threads', of warps four apart: half 0 has tokens 0 to 63 of each
    // block and the first half of O's columns, half 1 the others.
    const int t = warp >> 3, half = (warp >> 2) & 1;  // stream, half
    const int tt = (warp & 3) * 32 + lane;            // row in the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_sc = tmem + (uint32_t)t * kTok + 64 * half + lane_base;
    const uint32_t t_o = tmem + 256 + (uint32_t)t * D + (uint32_t)half * (D / 2) + lane_base;
    // 64 columns that hold nothing before the stream's first P is handed over
    const uint32_t t_free = D == 64 ? tmem + 384 + 64 * half + lane_base : t_o;
    float* const xch = reinterpret_cast<float*>(base_ptr + PL::kOffX) + t * 4 * kRows;
    // What both threads of a row bring, and whether all of the two warps go on.  Two
    // places in turn: nobody is more than one exchange ahead.
    int turn = 0;
    auto exchange = [&](float mine, bool good, float& its) -> bool {
      float* at = xch + turn * 2 * kRows + tt;
      turn ^= 1;
      at[half * kRows] = mine;
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.and.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(r) : "r"((uint32_t)good), "r"(2 + t * 4 + (warp & 3)) : "memory");
      its = at[(half ^ 1) * kRows];
      return r != 0;
    };
    bool cold = true;
    const float c2 = p.scale_log2;
    // A wait that gave up: the walk goes on for the exchanges, and nothing else.
    bool ok = true;
    int done = 0;            // blocks of the stream so far
    int u0 = 0, u1 = 0;      // uses of V's buffers so far
    for (int ln = 0; ln < 2; ++ln) {  // line 2, then the stream's share of line 1
      begin(ln == 0 ? 0 : 1 + t);
      // what the share leaves for the merge, if anything, is its last part
      const bool tells = tt == 0 && half == 0 && (ln == 1 || t == 0);
      if (tells) p.meta[2 * (ln == 0 ? wk.share : grid + wk.share)] = make_int4(0, 0, 0, 0);
      while (next()) {
        const int nt = wk.s.nblk;
        int tok0 = wk.s.j0 * kTok;
        const int row = wk.s.row0 + (two ? t * kRows : 0) + tt;  // node x g + head
        const bool real = row < wk.n * G;
        const bool busy = row - lane < wk.n * G;  // a warp without rows only keeps the barriers
        const int past = wk.ctx - wk.n;
        uint64_t mask = 0, any = 0;  // the nodes that the row sees, and that any row does
        float m_ref = -INFINITY, l_sum = 0.f;
        // The first part begins with a step on whatever lies in columns that no product
        // uses yet, and drops what comes out: it brings the instructions into the cache
        // while the first blocks are on their way (about 5000 cycles else).
        int i = cold ? -1 : 0;
        cold = false;
        if (i < 0) tok0 -= kTok;
        for (; i < nt; ++i, tok0 += kTok) {
          const int kb = two ? i & 1 : t;  // the block's buffers, and their uses before
          const int ku = (kb ? u1 : u0) + (two ? i >> 1 : i);
          const uint32_t t_s = i < 0 ? t_free : t_sc;
          if (i >= 0 && tok0 + kTok > past && (i == 0 || tok0 <= past)) {
            // the first block with nodes: their words come while the scores are on their
            // way (at the part's start they waited behind the last part's stores, 3000
            // cycles: ragged trees 90.5 us, then 88)
            const uint64_t nodes = wk.n == 64 ? ~0ull : (1ull << wk.n) - 1;
            if (real) mask = (uint64_t)p.tree_mask[wk.q0 + row / G] & nodes;
            any = lane < wk.n ? (uint64_t)p.tree_mask[wk.q0 + lane] : 0ull;
            if (lane + 32 < wk.n) any |= (uint64_t)p.tree_mask[wk.q0 + lane + 32];
            any = ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32)) << 32 |
                   __reduce_or_sync(0xffffffffu, (uint32_t)any)) & nodes;
          }
          if (i >= 0) {
            ok = ok && __all_sync(0xffffffffu, wait(kBarSFull + t, (uint32_t)((done + i) & 1)));
            tc_fence_after();
          }
          // a page outside the pool (reported by the copy warp, zeros in shared memory)
          // is left out: bit pg stands for the block's page pg
          const uint32_t bad = i < 0 ? 0 : bad_pages[2 * kb + (ku & 1)];
          if (busy) {
            uint32_t sa[16], sb[16];
            if (i >= 0 && (tok0 + kTok > past || bad != 0)) {  // scores that the row does not see
#pragma unroll 1
              for (int k = 0; k < 4; ++k) {  // a page
                const int pg = 4 * half + k;
                // bit e: whether the row sees token tok0 + 16 pg + e
                const int s = tok0 + kPageSize * pg - past;  // of node 0, negative in the past
                uint32_t v = s <= -16 ? 0xffffu : s >= 64 ? 0u : s >= 0 ? (uint32_t)(mask >> s)
                             : (uint32_t)(mask << -s) | ((1u << -s) - 1);
                if ((bad >> pg) & 1) v = 0;
                if (__all_sync(0xffffffffu, (v & 0xffffu) == 0xffffu)) continue;
                tmem_ld16_issue(t_s + 16 * k, sa);
                tmem_ld16_wait(sa);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (!((v >> e) & 1)) sa[e] = 0xff800000u;  // -inf
                tmem_st16_issue(t_s + 16 * k, sa);
                tmem_st_wait();
              }
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            auto smax = [&](const uint32_t (&s)[16]) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                m4[e & 3] =
                    max3(m4[e & 3], __uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
            };
            // 16 tokens at a time, from the last: the first are still in sa when P's turn
            // comes
            tmem_ld16_issue(t_s + 48, sb);
            tmem_ld16_wait(sb);
            tmem_ld16_issue(t_s + 32, sa);
            smax(sb);
            tmem_ld16_wait(sa);
            tmem_ld16_issue(t_s + 16, sb);
            smax(sa);
            tmem_ld16_wait(sb);
            tmem_ld16_issue(t_s, sa);
            smax(sb);
            tmem_ld16_wait(sa);
            smax(sa);
            float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), its;
            ok = exchange(mx, ok, its);
            mx = fmaxf(mx, its) * c2 - kRefBelow<BF16>;
            const bool grow = mx > m_ref + 8.f;  // lazy rescale, as in the prefill kernel
            float alpha = 1.f;
            if (grow) {
              alpha = ex2(m_ref - mx);
              m_ref = mx;
              l_sum *= alpha;
            }
            if (i > 0) {
              ok = ok &&
                   __all_sync(0xffffffffu, wait(kBarODone + t, (uint32_t)((done + i - 1) & 1)));
              tc_fence_after();
              if (ok && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
                for (int cc = 0; cc < D / 64; ++cc) {
                  uint32_t r[32];
                  tmem_ld32(t_o + (uint32_t)cc * 32, r);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                  tmem_st32(t_o + (uint32_t)cc * 32, r);
                }
              }
            }
            const float mu = m_ref == -INFINITY ? 0.f : m_ref;
            const uint64_t c2x2 = f2(c2, c2), nmu2 = f2(-mu, -mu);
            uint64_t acc[2] = {0ull, 0ull};
            // P of 16 tokens over their scores: eight columns of hi pairs, eight of lo pairs
            auto weigh = [&](const uint32_t (&s)[16], uint32_t c) {
              uint32_t pq[16];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 y = f2_split(fma2(f2(__uint_as_float(s[2 * e]),
                                                  __uint_as_float(s[2 * e + 1])), c2x2, nmu2));
                const float p0 = ex2(y.x), p1 = ex2(y.y);
                const uint64_t pp = f2(p0, p1);
                acc[e & 1] = add2(acc[e & 1], pp);
                pq[e] = pack2<BF16>(p0, p1);
                const float2 hf = floats_of<BF16>(pq[e]);
                const float2 l = f2_split(sub2(pp, f2(hf.x, hf.y)));
                pq[8 + e] = pack2<BF16>(l.x, l.y);
              }
              tmem_st16_issue(t_s + c, pq);
            };
            tmem_ld16_issue(t_s + 16, sb);
            weigh(sa, 0);
            tmem_ld16_wait(sb);
            tmem_ld16_issue(t_s + 32, sa);
            weigh(sb, 16);
            tmem_ld16_wait(sa);
            tmem_ld16_issue(t_s + 48, sb);
            weigh(sa, 32);
            tmem_ld16_wait(sb);
            weigh(sb, 48);
            tmem_st_wait();
            const float2 a0 = f2_split(add2(acc[0], acc[1]));
            l_sum += a0.x + a0.y;
          }
          if (i < 0) {
            m_ref = -INFINITY;
            l_sum = 0.f;
            continue;
          }
          // V rows behind the end, and of nodes that no row sees, may hold anything
          // (0 x NaN): zeroed in the staged block by the stream that uses it first
          if (tok0 + kTok > past && (t == 0 || !two)) {
            ok = ok && __all_sync(0xffffffffu, wait(kBarVFull + kb, (uint32_t)(ku & 1)));
            const int first = max(0, past - tok0);
            const uint32_t vb = base + kOffV + (uint32_t)kb * NH * kHalf;
            for (int e = half * kRows + tt; ok && e < (kTok - first) * 8 * NH; e += kSoft) {
              const int rr = first + e / (8 * NH), ch = e % (8 * NH), node = tok0 + rr - past;
              if (node < wk.n && ((any >> node) & 1)) continue;
              const uint32_t a = vb + (uint32_t)(ch >> 3) * kHalf + (uint32_t)rr * 128 +
                                 (uint32_t)(ch & 7) * 16;
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
            }
            // the tensor cores read them through the async proxy
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          tc_fence_before();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(bar(kBarPFull + t));
        }
        // ---- the part's end: the row's output, or the part's m, l and unnormalised o
        ok = ok && __all_sync(0xffffffffu, wait(kBarODone + t, (uint32_t)((done + nt - 1) & 1)));
        done += nt;
        u0 += two ? (nt + 1) / 2 : nt;
        u1 += two ? nt / 2 : nt;
        const bool head = wk.s.j0 > 0, ends = wk.s.j0 + nt == wk.s.total, whole = !head && ends;
        if (tells && !whole && !head) {  // the shares that hold the rest follow this one
          const int64_t cost = line[p.B];
          const int64_t shares = tree_shares(cost, two ? grid : 2 * grid);
          const int parts = (int)tree_share_of(wk.at - kTreeBlock, cost, shares) - wk.share + 1;
          const int64_t o = (int64_t)(wk.q0 + wk.s.row0 / G) * p.Hq + wk.s.h * G;
          // parts, rows; the output row of the first
          int4* const meta = p.meta + 2 * (ln == 0 ? wk.share : grid + wk.share);
          meta[0] = make_int4(parts, min(two ? 2 * kRows : kRows, wk.n * G - wk.s.row0), 0, 0);
          meta[1] = make_int4((int)(o & 0xffffffff), (int)(o >> 32), 0, 0);
        }
        if (busy) {
          float its;
          ok = exchange(l_sum, ok, its);
          l_sum = half == 0 ? l_sum + its : its + l_sum;  // the same sum in both
        }
        if (ok && busy) {
          tc_fence_after();
          const bool some = l_sum != 0.f;  // NaN counts: it has to show
          const int64_t prow =
              (2 * (int64_t)wk.share + (head ? 0 : 1)) * (two ? 2 * kRows : kRows) +
              (two ? t * kRows : 4 * kRows * (int64_t)grid) + tt;
          float* const po = p.part_o + part_at<D>(prow) + half * (D / 16) * kPartStep;
          const float inv = some ? 1.f / l_sum : 0.f;
          const int64_t orow = (int64_t)(wk.q0 + row / G) * p.Hq + wk.s.h * G + row % G;
          if (!whole && real && half == 0)
            p.part_ml[prow] = some ? make_float2(m_ref, l_sum) : make_float2(-INFINITY, 0.f);
#pragma unroll 1
          for (int cc = 0; cc < D / 64; ++cc) {
            uint32_t r[32];
            tmem_ld32(t_o + (uint32_t)cc * 32, r);
            if (!real) continue;
            const int col = half * (D / 2) + cc * 32;
            if (!whole) {
#pragma unroll
              for (int e = 0; e < 4; ++e) store32(po + (4 * cc + e) * kPartStep, r + 8 * e);
              continue;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * inv);
            uint4* to;  // (the output need not be aligned to whole sectors)
            if (p.out_dtype == PKV_F32) {
              to = reinterpret_cast<uint4*>(static_cast<float*>(p.out) + orow * D + col);
#pragma unroll
              for (int e = 4; e < 8; ++e)
                to[e] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
            } else {
              to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + orow * D + col);
              const bool bf = p.out_dtype == PKV_BF16;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float x = __uint_as_float(r[2 * e]), y = __uint_as_float(r[2 * e + 1]);
                r[e] = bf ? pack2<true>(x, y) : pack2<false>(x, y);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              to[e] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
          }
          tc_fence_before();  // O_t is read before P_t of the next part is handed over
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

// ---- the merge of the segments that share boundaries cut.  Every CTA lists them
// (their groups of rows, summed up) and its warps take every grid-th group.  Eight
// lanes hold a row's columns: a warp joins four rows of a segment with few parts, or
// the parts of one row of a segment with many, every fourth in eight lanes; four parts
// are in flight per lane.  Bound by latency: the launch, a round of loads, and the code,
// which is fetched anew by every launch and therefore short (four rows per warp and lane
// unrolled took 22 us for 35 MB of partials).  One CTA per SM, so that a thread has 128
// registers: two with 64, whose loads spilled, took ragged trees of 32 sequences from 83
// to 87.5 us and one sequence of 32768 tokens from 36 to 42.
constexpr int kMergeThreads = 512, kMergeWarps = kMergeThreads / 32;
constexpr int kMergeAt = 4;
// Whether a row's parts are spread over a warp: more than four of a segment with few
// rows, whose warps would else be few, or more than eight (64 nodes behind 701 tokens,
// 224 rows in 6 parts: 16.8 us with four for all, 15.7; 28 rows: 11.0 with eight, 10.7).
__device__ __forceinline__ bool merge_many(int parts, int rows) {
  return parts > (rows > 32 ? 8 : 4);
}
constexpr int kMergeShares = 768;  // room for the shares of both lines
constexpr int kMaxCtas = kMergeShares / 3;

template <int D>
__global__ void __launch_bounds__(kMergeThreads, 1) tree_merge_kernel(const TreeParams p) {
  __shared__ int upto[kMergeShares];   // groups up to and with a cut segment
  __shared__ int4 cut[kMergeShares];   // its entry of meta, parts and rows, first output row
  __shared__ int warp_n[kMergeWarps], warp_g[kMergeWarps];
  griddep_wait_then_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int cuts = 0, groups = 0;
  for (int i0 = 0; i0 < 3 * p.ctas; i0 += kMergeThreads) {
    const int i = i0 + tid;
    int4 m = make_int4(0, 0, 0, 0), o = m;
    if (i < 3 * p.ctas) {
      m = p.meta[2 * i];
      o = p.meta[2 * i + 1];
    }
    const int mine = m.x == 0 ? 0 : merge_many(m.x, m.y) ? m.y : (m.y + kMergeAt - 1) / kMergeAt;
    int g = mine;  // groups up to this entry's
#pragma unroll
    for (int o2 = 1; o2 < 32; o2 <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, g, o2);
      if (lane >= o2) g += v;
    }
    const uint32_t any = __ballot_sync(0xffffffffu, mine > 0);
    if (lane == 31) {
      warp_g[warp] = g;
      warp_n[warp] = __popc(any);
    }
    __syncthreads();
    const int wn = lane < kMergeWarps ? warp_n[lane] : 0, wg = lane < kMergeWarps ? warp_g[lane] : 0;
    const int at = cuts + __reduce_add_sync(0xffffffffu, lane < warp ? wn : 0) +
                   __popc(any & ((1u << lane) - 1));
    g += groups + __reduce_add_sync(0xffffffffu, lane < warp ? wg : 0);
    cuts += __reduce_add_sync(0xffffffffu, wn);
    groups += __reduce_add_sync(0xffffffffu, wg);
    if (mine > 0) {
      upto[at] = g;
      cut[at] = make_int4(i | m.y << 16, m.x, o.x, o.y);
    }
    __syncthreads();
  }
  constexpr int V = D / 32;  // groups of four columns of a lane
  // group g of warp w of CTA c is w grid + c: a segment's rows spread over the SMs
  for (int g = warp * gridDim.x + blockIdx.x; g < groups; g += gridDim.x * kMergeWarps) {
    int a = 0;  // the first cut segment whose sum is above g
    for (int z = cuts - 1; a < z;) {
      const int mid = (a + z) >> 1;
      if (upto[mid] > g) z = mid; else a = mid + 1;
    }
    const int4 m = cut[a];
    const int i = m.x & 0xffff, rows = m.x >> 16, parts = m.y;
    const int sub = g - (a > 0 ? upto[a - 1] : 0);
    const bool two = i < p.ctas;
    const int c = two ? i : i - p.ctas, per = two ? 2 * kRows : kRows;
    const int64_t out0 = (int64_t)(uint32_t)m.z | (int64_t)m.w << 32;
    // the parts: slot 2 c + 1, then 2 c' of the shares behind
    const int64_t first = two ? 0 : 4 * kRows * (int64_t)p.ctas;
    auto slot = [&](int k) -> int64_t {
      return first + (k == 0 ? 2 * (int64_t)c + 1 : 2 * (int64_t)(c + k)) * per;
    };
    const bool many = merge_many(parts, rows);
    const int row = many ? sub : sub * kMergeAt + (lane >> 3);
    const bool real = row < rows;
    // against a running maximum, so that m, l and o of a part are loaded together
    float M = -INFINITY, l = 0.f, acc[4 * V];
#pragma unroll
    for (int e = 0; e < 4 * V; ++e) acc[e] = 0.f;
    auto down = [&](float m2) -> float {  // to the new reference; the factor of a part at m2
      const float top = fmaxf(M, m2), ref = top == -INFINITY ? 0.f : top;
      const float w = ex2(M - ref);
      M = top;
      l *= w;
#pragma unroll
      for (int e = 0; e < 4 * V; ++e) acc[e] *= w;
      return ex2(m2 - ref);
    };
    const int step = many ? 4 : 1;
    const float* mine = p.part_o + ((lane & 7) >> 1) * kPartStep + 4 * (lane & 1);  // of a row
#pragma unroll 1
    for (int k = many ? lane >> 3 : 0; real && k < parts; k += 4 * step) {
      float2 ml[4];
      float4 x[4][V];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        if (k + f * step >= parts) break;
        const int64_t at = slot(k + f * step) + row;
        ml[f] = p.part_ml[at];
#pragma unroll
        for (int e = 0; e < V; ++e)
          x[f][e] = *reinterpret_cast<const float4*>(mine + part_at<D>(at) + 4 * e * kPartStep);
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        if (k + f * step >= parts) break;
        if (ml[f].y == 0.f) continue;  // a part with nothing in it, whose o holds anything
        const float w = down(ml[f].x);
        l += w * ml[f].y;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          acc[4 * e] += w * x[f][e].x;
          acc[4 * e + 1] += w * x[f][e].y;
          acc[4 * e + 2] += w * x[f][e].z;
          acc[4 * e + 3] += w * x[f][e].w;
        }
      }
    }
    if (many) {
#pragma unroll 1
      for (int o = 8; o < 32; o <<= 1) {
        down(__shfl_xor_sync(0xffffffffu, M, o));  // both lanes, to the same reference
        l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
        for (int e = 0; e < 4 * V; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
      }
    }
    if (!real || (many && lane >= 8)) continue;
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int G = p.Hq / p.Hkv;
    const int64_t to = (out0 + (int64_t)(row / G) * p.Hq + row % G) * D + 4 * (lane & 7);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float4 y = make_float4(acc[4 * e] * inv, acc[4 * e + 1] * inv, acc[4 * e + 2] * inv,
                                   acc[4 * e + 3] * inv);
      if (p.out_dtype == PKV_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to + 32 * e) = y;
      } else {
        const bool bf = p.out_dtype == PKV_BF16;
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + to + 32 * e) =
            make_uint2(bf ? pack2<true>(y.x, y.y) : pack2<false>(y.x, y.y),
                       bf ? pack2<true>(y.z, y.w) : pack2<false>(y.z, y.w));
      }
    }
  }
}

static_assert(kMaxCtas >= kTreeMaxCtas, "the merge lists every share");

template <bool BF16, int D>
cudaError_t launch(const TreeLaunch& l) {
  auto kern = tree_kernel<BF16, D>;
  static std::atomic<uint64_t> configured{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Plan<D>::smem(kTreeMaxBatch));
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  e = launch_dependent(kern, dim3((unsigned)l.p.ctas), dim3(kThreads), Plan<D>::smem(l.p.B),
                       l.stream, l.p, l.tmap_q, l.tmap_k, l.tmap_v);
  if (e != cudaSuccess) return e;
  return launch_dependent(tree_merge_kernel<D>, dim3((unsigned)l.p.ctas),
                          dim3(kMergeThreads), 0, l.stream, l.p);
}

}  // namespace tr

cudaError_t launch_tree(const TreeLaunch& l) {
  if (l.d == 64) return l.bf16 ? tr::launch<true, 64>(l) : tr::launch<false, 64>(l);
  if (l.d == 128) return l.bf16 ? tr::launch<true, 128>(l) : tr::launch<false, 128>(l);
  return cudaErrorNotSupported;
}

}  // namespace pkv
