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
//   warps 0-3, 4-7  softmax of stream 0, 1: one row per thread, TMEM lane t;
//   warps 8, 11     issue the MMAs; warps 9, 10 the tensor copies.
// A stream is a row tile with its accumulator.
//   Line 2, segments of two tiles: a share per CTA.  Both streams take every
//   block, K and V double-buffered and copied by a warp each; warp 8 issues.
//   Line 1, segments of one tile (up to 128 rows: the usual tree), after it: a
//   share per stream, with a K and a V buffer, a copying and an issuing warp of
//   its own, so that one stream's segment ends, copies and products run under the
//   other's softmax.
//   S = Q K^T   tcgen05.mma M 128 x N 128 x K d from shared memory;
//   P           hi + lo 16-bit pairs over S in tensor memory;
//   O += P V    tcgen05.mma with A from tensor memory, twice per 16 tokens.
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
constexpr int kThreads = 384;
constexpr uint32_t kHalf = 16384;  // 128 rows x 128 bytes: 64 d columns of a tile or block
// one barrier per buffer or stream, in pairs
constexpr int kBarQ = 0, kBarQFree = 2, kBarKFull = 4, kBarVFull = 6, kBarKFree = 8,
              kBarVFree = 10, kBarSFull = 12, kBarPFull = 14, kBarODone = 16, kNumBars = 18;
constexpr uint32_t kTmemCols = 512;  // S0/P0, S1/P1, then O0, O1
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kSeqs = 128;  // sequences whose rows and lengths are at hand in shared memory

template <int D>
struct Plan {
  static constexpr int NH = D / 64;
  static constexpr uint32_t kOffK = 2 * NH * kHalf;
  static constexpr uint32_t kOffV = 4 * NH * kHalf;
  static constexpr uint32_t kOffBar = 6 * NH * kHalf;
  static constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;     // TMEM base, abort, counts
  static constexpr uint32_t kOffSeq = (kOffMisc + 24 + 4 * kNumBars + 15) / 16 * 16;  // [kSeqs]
  static constexpr uint32_t kOffPfx = kOffSeq + 16 * kSeqs;  // [2][B+1]
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
  uint32_t* pfx = reinterpret_cast<uint32_t*>(base_ptr + PL::kOffPfx);  // [2][B+1] costs before

  if (tid == 0) {
    prefetch_tmap(&tmq);
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
    *abort_flag = 0;
    for (int i = 0; i < kNumBars; ++i) {
      armed[i] = 0;
      mbar_init(bar(i), (i == kBarPFull || i == kBarPFull + 1) ? kRows / 32 : 1);
    }
    fence_mbar_init();
    pfx[0] = 0;
    pfx[p.B + 1] = 0;
  }
  // so far nothing of the kernel in front was needed, and it may still run
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  auto begin = [&](bool t2, int share, int most) {  // of `most` shares at most
    two = t2;
    line = pfx + (t2 ? p.B + 1 : 0);
    const int64_t cost = line[p.B], n = tree_shares(cost, most);
    wk.share = share;
    wk.at = share < n ? (uint32_t)tree_share(share, cost, n) : 0;
    wk.hi = share < n ? (uint32_t)tree_share(share + 1, cost, n) : 0;
    int a = 0;  // the sequence holding `at`: the last with line <= at
    if (wk.at < wk.hi) {
      for (int z = p.B; z - a > 1;) {
        const int mid = (a + z) >> 1;
        if (line[mid] <= wk.at) a = mid; else z = mid;
      }
    }
    wk.s.b = a;
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
  const int grid = gridDim.x;
  auto begin2 = [&]() { begin(true, blockIdx.x, grid); };
  // the first shares of line 1 go to CTAs of their own
  auto begin1 = [&](int t) { begin(false, t * grid + blockIdx.x, 2 * grid); };

  auto wait = [&](int i, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(i), parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait_bounded(bar(i), parity, kWaitNs)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp == 9 || warp == 10) {
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
    const bool v = warp == 10;
    begin2();  // warp 9: Q and K, warp 10: V
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
    const int t = warp - 9;
    begin1(t);  // each a stream
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
  } else if (warp == 8 || warp == 11) {
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
      // The first product over O_t of a part comes after P_t, which the softmax
      // threads hand over after they have read the last part's O_t out.
      if (elect_one()) {
        begin2();
        while (ok && next()) {  // one buffer after the other, both streams from it
          const int n = wk.s.nblk;
          if (warp == 8) {  // (warp 11 counts)
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
      // Then a stream each, whose products are a chain.  Warp 11 begins when warp 8
      // has issued all of line 2 (no earlier: a barrier's phases are told apart by
      // parity) and stream 1's last product of it, which is another thread's, is done.
      __syncwarp();
      asm volatile("bar.sync 1, 64;" ::: "memory");
      if (elect_one()) {  // the lane that was elected before
        const int t = warp == 11;
        uint32_t u = t ? u1 : u0;
        if (t == 1 && st > 0) {
          ok = wait(kBarODone + 1, (st - 1) & 1);
          tc_fence_after();
        }
        begin1(t);
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
    const int t = warp >> 2;           // stream
    const int tt = tid - t * kRows;    // row in the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + (uint32_t)t * kTok + lane_base;
    const uint32_t t_o = tmem + 256 + (uint32_t)t * D + lane_base;
    const float c2 = p.scale_log2;
    bool ok = true;
    int done = 0;            // blocks of the stream so far
    int u0 = 0, u1 = 0;      // uses of V's buffers so far
    // what the share leaves for the merge: parts (0: nothing), rows; the output row of
    // the first (as two words)
    int4 left = make_int4(0, 0, 0, 0), left_at = left;
    for (int ln = 0; ln < 2; ++ln) {  // line 2, then the stream's share of line 1
    if (ln == 0) begin2();
    else begin1(t);
    while (ok && next()) {
      const int nt = wk.s.nblk;
      int tok0 = wk.s.j0 * kTok;
      const int row = wk.s.row0 + (two ? t * kRows : 0) + tt;  // node x g + head
      const bool real = row < wk.n * G;
      const bool busy = row - lane < wk.n * G;  // a warp without rows only keeps the barriers
      const int past = wk.ctx - wk.n;
      // the nodes that the row sees, and those that any row of the tree does
      const uint64_t nodes = wk.n == 64 ? ~0ull : (1ull << wk.n) - 1;
      uint64_t mask = real ? (uint64_t)p.tree_mask[wk.q0 + row / G] & nodes : 0ull;
      uint64_t any = lane < wk.n ? (uint64_t)p.tree_mask[wk.q0 + lane] : 0ull;
      if (lane + 32 < wk.n) any |= (uint64_t)p.tree_mask[wk.q0 + lane + 32];
      any = ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32)) << 32 |
             __reduce_or_sync(0xffffffffu, (uint32_t)any)) & nodes;
      float m_ref = -INFINITY, l_sum = 0.f;
      for (int i = 0; ok && i < nt; ++i, tok0 += kTok) {
        const int kb = two ? i & 1 : t;  // the block's buffers, and their uses before
        const int ku = (kb ? u1 : u0) + (two ? i >> 1 : i);
        ok = __all_sync(0xffffffffu, wait(kBarSFull + t, (uint32_t)((done + i) & 1)));
        if (!ok) break;
        tc_fence_after();
        // a page outside the pool (reported by the copy warp, zeros in shared memory)
        // is left out: bit pg stands for the block's page pg
        const uint32_t bad = bad_pages[2 * kb + (ku & 1)];
        if (busy) {
        uint32_t sa[32], sb[32];
        if (tok0 + kTok > past || bad != 0) {  // scores that the row does not see
#pragma unroll 1
          for (int qq = 0; qq < 4; ++qq) {
            // bit e: whether the row sees token tok0 + 32 qq + e
            const int s = tok0 + 32 * qq - past;  // of the tree's node 0, negative in the past
            uint32_t v = s <= -32 ? 0xffffffffu : s >= 64 ? 0u : s >= 0 ? (uint32_t)(mask >> s)
                         : (uint32_t)(mask << -s) | ((1u << -s) - 1);
            if ((bad >> (2 * qq)) & 1) v &= 0xffff0000u;
            if ((bad >> (2 * qq + 1)) & 1) v &= 0x0000ffffu;
            if (__all_sync(0xffffffffu, v == 0xffffffffu)) continue;
            tmem_ld32(t_s + 32 * qq, sa);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((v >> e) & 1)) sa[e] = 0xff800000u;  // -inf
            tmem_st32(t_s + 32 * qq, sa);
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto qmax = [&](const uint32_t (&sq)[32]) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            m4[e & 3] = max3(m4[e & 3], __uint_as_float(sq[2 * e]), __uint_as_float(sq[2 * e + 1]));
        };
        // quarters 3, 2, 1, 0: quarter 0 is still in sb when the P pass starts
        tmem_ld32_issue(t_s + 96, sa);
        tmem_ld_wait(sa);
        tmem_ld32_issue(t_s + 64, sb);
        qmax(sa);
        tmem_ld_wait(sb);
        tmem_ld32_issue(t_s + 32, sa);
        qmax(sb);
        tmem_ld_wait(sa);
        tmem_ld32_issue(t_s + 0, sb);
        qmax(sa);
        tmem_ld_wait(sb);
        qmax(sb);
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c2;
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
            uint32_t r[32];
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
        uint32_t hi16[16], lo16[16];
        auto qp = [&](const uint32_t (&sq)[32]) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = f2_split(fma2(f2(__uint_as_float(sq[2 * e]),
                                              __uint_as_float(sq[2 * e + 1])), c2x2, nmu2));
            const float p0 = ex2(y.x), p1 = ex2(y.y);
            const uint64_t pp = f2(p0, p1);
            acc[e & 3] = add2(acc[e & 3], pp);
            hi16[e] = pack2<BF16>(p0, p1);
            const float2 hf = unpack2<BF16>(hi16[e]);
            const float2 l = f2_split(sub2(pp, f2(hf.x, hf.y)));
            lo16[e] = pack2<BF16>(l.x, l.y);
          }
        };
        auto qst = [&](int qq) {
          const uint32_t c = (uint32_t)(64 * (qq >> 1) + 16 * (qq & 1));
          tmem_st16_issue(t_s + c, hi16);
          tmem_st16_issue(t_s + c + 32, lo16);
        };
        tmem_ld32_issue(t_s + 32, sa);
        qp(sb);
        tmem_ld_wait(sa);
        qst(0);
        tmem_ld32_issue(t_s + 64, sb);
        qp(sa);
        tmem_ld_wait(sb);
        qst(1);
        tmem_ld32_issue(t_s + 96, sa);
        qp(sb);
        tmem_ld_wait(sa);
        qst(2);
        qp(sa);
        qst(3);
        tmem_st_wait();
        {
          const float2 a0 = f2_split(add2(acc[0], acc[1])), a1 = f2_split(add2(acc[2], acc[3]));
          l_sum += (a0.x + a0.y) + (a1.x + a1.y);
        }
        }
        // V rows behind the end, and of nodes that no row sees, may hold anything
        // (0 x NaN): zeroed in the staged block by the stream that uses it first
        if (tok0 + kTok > past && (t == 0 || !two)) {
          ok = __all_sync(0xffffffffu, wait(kBarVFull + kb, (uint32_t)(ku & 1)));
          if (!ok) break;
          const int first = max(0, past - tok0);
          const uint32_t vb = base + kOffV + (uint32_t)kb * NH * kHalf;
          for (int e = tt; e < (kTok - first) * 8 * NH; e += kRows) {
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
        if (lane == 0) mbar_arrive(bar(kBarPFull + t));
      }
      // ---- the part's end: the row's output, or the part's m, l and unnormalised o
      if (ok)
        ok = __all_sync(0xffffffffu, wait(kBarODone + t, (uint32_t)((done + nt - 1) & 1)));
      done += nt;
      u0 += two ? (nt + 1) / 2 : nt;
      u1 += two ? nt / 2 : nt;
      const bool head = wk.s.j0 > 0, ends = wk.s.j0 + nt == wk.s.total, whole = !head && ends;
      if (!whole) {
        if (!head) {  // the shares that hold the rest follow this one
          const int64_t cost = line[p.B];
          left.x = (int)tree_share_of(wk.at - kTreeBlock, cost,
                                      tree_shares(cost, two ? grid : 2 * grid)) - wk.share + 1;
          left.y = min(two ? 2 * kRows : kRows, wk.n * G - wk.s.row0);
          const int64_t o = (int64_t)(wk.q0 + wk.s.row0 / G) * p.Hq + wk.s.h * G;
          left_at.x = (int)(o & 0xffffffff);
          left_at.y = (int)(o >> 32);
        }
      }
      if (ok && busy) {
        tc_fence_after();
        const bool some = l_sum != 0.f;  // NaN counts: it has to show
        const int64_t prow = (2 * (int64_t)wk.share + (head ? 0 : 1)) * (two ? 2 * kRows : kRows) +
                             (two ? t * kRows : 4 * kRows * (int64_t)grid) + tt;
        const float inv = some ? 1.f / l_sum : 0.f;
        const int64_t orow = (int64_t)(wk.q0 + row / G) * p.Hq + wk.s.h * G + row % G;
        if (!whole && real)
          p.part_ml[prow] = some ? make_float2(m_ref, l_sum) : make_float2(-INFINITY, 0.f);
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t r[32];
          tmem_ld32(t_o + (uint32_t)cc * 32, r);
          if (!real) continue;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * inv);
            if (p.out_dtype != PKV_F32) {
              const bool bf = p.out_dtype == PKV_BF16;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float x = __uint_as_float(r[2 * e]), y = __uint_as_float(r[2 * e + 1]);
                r[e] = bf ? pack2<true>(x, y) : pack2<false>(x, y);
              }
              uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + orow * D +
                                                   cc * 32);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                to[e] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
              continue;
            }
          }
          float* po = whole ? static_cast<float*>(p.out) + orow * D + cc * 32
                            : p.part_o + prow * D + cc * 32;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reinterpret_cast<uint4*>(po)[e] =
                make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
        }
        tc_fence_before();  // O_t is read before P_t of the next part is handed over
      }
    }
    if (tt == 0 && (ln == 1 || t == 0)) {
      int4* meta = p.meta + 2 * (ln == 0 ? wk.share : grid + wk.share);
      meta[0] = left;
      meta[1] = left_at;
    }
    left.x = 0;
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
// (their groups of rows, summed up) and its warps take every grid-th group: a row
// of a segment with many parts, eight parts in flight, or kMergeAt rows of one with
// few.  (A grid over shares and rows, mostly empty, took 35 us, cold, for the
// case of 32 ragged sequences.)
constexpr int kMergeWarps = 8, kMergeAt = 4, kMergeFew = 4;
constexpr int kMergeShares = 1024;  // room for the shares of both lines

// kAt rows from r0 on of a segment by one warp, kFly parts in flight.
template <int D, int kAt, int kFly, typename Slot>
__device__ __forceinline__ void merge_rows(const TreeParams& p, Slot slot, int parts, int r0,
                                           int rows, int64_t out0) {
  constexpr int V = D / 32;  // columns per lane
  const int lane = threadIdx.x & 31;
  float M[kAt], acc[kAt][V], l[kAt];
  bool in[kAt];
#pragma unroll
  for (int a = 0; a < kAt; ++a) {
    in[a] = r0 + a < rows;
    l[a] = 0.f;
    M[a] = -INFINITY;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[a][e] = 0.f;
  }
  auto ml_of = [&](int k, int a) -> float2 {
    return in[a] && k < parts ? p.part_ml[slot(k) + r0 + a]
                              : make_float2(-INFINITY, 0.f);
  };
  float2 ml[kAt];
  for (int k0 = 0; k0 < parts; k0 += 32) {
#pragma unroll
    for (int a = 0; a < kAt; ++a) {
      ml[a] = ml_of(k0 + lane, a);
      M[a] = fmaxf(M[a], ml[a].x);
    }
  }
#pragma unroll
  for (int a = 0; a < kAt; ++a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M[a] = fmaxf(M[a], __shfl_xor_sync(0xffffffffu, M[a], o));
    if (M[a] == -INFINITY) M[a] = 0.f;  // nothing at all, or nothing but NaN
  }
  for (int k0 = 0; k0 < parts; k0 += 32) {
    if (parts > 32) {  // else they are at hand
#pragma unroll
      for (int a = 0; a < kAt; ++a) ml[a] = ml_of(k0 + lane, a);
    }
    for (int k1 = k0; k1 < k0 + 32 && k1 < parts; k1 += kFly) {
      float x[kFly][kAt][V];
#pragma unroll
      for (int f = 0; f < kFly; ++f)
#pragma unroll
        for (int a = 0; a < kAt; ++a) {
          const float lk = __shfl_sync(0xffffffffu, ml[a].y, k1 + f - k0);
#pragma unroll
          for (int e = 0; e < V; ++e) x[f][a][e] = 0.f;
          if (k1 + f >= parts || lk == 0.f) continue;  // a part with nothing in it
          const float* from = p.part_o + (slot(k1 + f) + r0 + a) * D + lane * V;
          if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4*>(from);
            x[f][a][0] = v.x;
            x[f][a][1] = v.y;
            x[f][a][2] = v.z;
            x[f][a][3] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(from);
            x[f][a][0] = v.x;
            x[f][a][1] = v.y;
          }
        }
#pragma unroll
      for (int f = 0; f < kFly; ++f)
#pragma unroll
        for (int a = 0; a < kAt; ++a) {
          const float mk = __shfl_sync(0xffffffffu, ml[a].x, k1 + f - k0);
          const float lk = __shfl_sync(0xffffffffu, ml[a].y, k1 + f - k0);
          const float w = k1 + f < parts ? ex2(mk - M[a]) : 0.f;
          l[a] += w * lk;
#pragma unroll
          for (int e = 0; e < V; ++e) acc[a][e] += w * x[f][a][e];
        }
    }
  }
#pragma unroll
  for (int a = 0; a < kAt; ++a) {
    if (!in[a]) continue;
    const float inv = l[a] != 0.f ? 1.f / l[a] : 0.f;
    const int G = p.Hq / p.Hkv, row = r0 + a;
    const int64_t to = (out0 + (int64_t)(row / G) * p.Hq + row % G) * D + lane * V;
    if (p.out_dtype == PKV_F32) {
#pragma unroll
      for (int e = 0; e < V; ++e) static_cast<float*>(p.out)[to + e] = acc[a][e] * inv;
    } else {
      const bool bf = p.out_dtype == PKV_BF16;
      uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + to);
#pragma unroll
      for (int e = 0; e < V / 2; ++e)
        out[e] = bf ? pack2<true>(acc[a][2 * e] * inv, acc[a][2 * e + 1] * inv)
                    : pack2<false>(acc[a][2 * e] * inv, acc[a][2 * e + 1] * inv);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const TreeParams p) {
  __shared__ int upto[kMergeShares];      // groups up to and with a cut segment
  __shared__ int16_t share[kMergeShares]; // its entry in meta
  __shared__ int warp_n[kMergeWarps], warp_g[kMergeWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int cuts = 0, groups = 0;
  for (int i0 = 0; i0 < 3 * p.ctas; i0 += kMergeWarps * 32) {
    const int i = i0 + tid;
    const int4 m = i < 3 * p.ctas ? p.meta[2 * i] : make_int4(0, 0, 0, 0);
    const int mine = m.x == 0 ? 0 : m.x > kMergeFew ? m.y : (m.y + kMergeAt - 1) / kMergeAt;
    int g = mine;  // groups up to this entry's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, g, o);
      if (lane >= o) g += v;
    }
    const uint32_t any = __ballot_sync(0xffffffffu, mine > 0);
    if (lane == 31) {
      warp_g[warp] = g;
      warp_n[warp] = __popc(any);
    }
    __syncthreads();
    int at = cuts + __popc(any & ((1u << lane) - 1));
    g += groups;
    for (int w = 0; w < kMergeWarps; ++w) {
      if (w < warp) {
        at += warp_n[w];
        g += warp_g[w];
      }
      cuts += warp_n[w];
      groups += warp_g[w];
    }
    if (mine > 0) {
      upto[at] = g;
      share[at] = (int16_t)i;
    }
    __syncthreads();
  }
  for (int g = blockIdx.x * kMergeWarps + warp; g < groups; g += gridDim.x * kMergeWarps) {
    int a = 0;  // the first cut segment whose sum is above g
    for (int z = cuts - 1; a < z;) {
      const int mid = (a + z) >> 1;
      if (upto[mid] > g) z = mid; else a = mid + 1;
    }
    const int i = share[a], sub = g - (a > 0 ? upto[a - 1] : 0);
    const int4 m = p.meta[2 * i], o = p.meta[2 * i + 1];
    const bool two = i < p.ctas;
    const int c = two ? i : i - p.ctas, per = two ? 2 * kRows : kRows;
    const int64_t out0 = (int64_t)(uint32_t)o.x | (int64_t)o.y << 32;
    // the parts: slot 2 c + 1, then 2 c' of the shares behind
    const int64_t first = two ? 0 : 4 * kRows * (int64_t)p.ctas;
    auto slot = [&](int k) -> int64_t {
      return first + (k == 0 ? 2 * (int64_t)c + 1 : 2 * (int64_t)(c + k)) * per;
    };
    if (m.x > kMergeFew) merge_rows<D, 1, 8>(p, slot, m.x, sub, m.y, out0);
    else merge_rows<D, kMergeAt, 2>(p, slot, m.x, sub * kMergeAt, m.y, out0);
  }
}

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
  return launch_dependent(tree_merge_kernel<D>, dim3((unsigned)(2 * l.p.ctas)),
                          dim3(kMergeWarps * 32), 0, l.stream, l.p);
}

}  // namespace tr

cudaError_t launch_tree(const TreeLaunch& l) {
  if (l.d == 64) return l.bf16 ? tr::launch<true, 64>(l) : tr::launch<false, 64>(l);
  if (l.d == 128) return l.bf16 ? tr::launch<true, 128>(l) : tr::launch<false, 128>(l);
  return cudaErrorNotSupported;
}

}  // namespace pkv
