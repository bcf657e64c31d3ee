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
// tree_kernel.  Persistent, at most one CTA per SM; the segments (sequence, pair
// of 128-row tiles, KV head) lie on one line of costs, cut into equal shares (see
// pkv_tree_line.h), so that ragged contexts and one long one both fill the GPU.
// A segment wholly inside a share is normalised and written at once; one that is
// cut leaves a partial in each CTA: slot 2 c where it came from the CTA before,
// 2 c + 1 where it starts in c.  Roles hand over through mbarriers:
//   warps 0-3, 4-7  softmax of stream 0, 1: one row per thread, TMEM lane t;
//   warp 8          issues the MMAs; warp 9 the copies of Q and K, warp 10 those of V.
// A stream is a row tile with its accumulator.  Two tiles share every block (K
// and V double-buffered).  Where a pair has one tile (up to 128 rows: the usual
// tree), both streams are that tile, stream t taking every second block in
// buffer t, so that one stream's products and copies run under the other's
// softmax; at a segment's end the threads of both streams exchange (m, l) and
// each joins half the columns of the two accumulators.
//   S = Q K^T   tcgen05.mma M 128 x N 128 x K d from shared memory;
//   P           hi + lo 16-bit pairs over S in tensor memory;
//   O += P V    tcgen05.mma with A from tensor memory, twice per 16 tokens.
//
// tree_merge_kernel.  A warp per row of a cut segment joins its parts, in order.
#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"
#include "pkv_tree_line.h"

namespace pkv {
namespace tr {

constexpr int kRows = kTreeRows, kTok = kTreeTok;
constexpr int kPages = kTok / kPageSize;
constexpr int kThreads = 352;
constexpr uint32_t kHalf = 16384;  // 128 rows x 128 bytes: 64 d columns of a tile or block
// one barrier per buffer or stream, in pairs
constexpr int kBarQ = 0, kBarQFree = 2, kBarKFull = 4, kBarVFull = 6, kBarKFree = 8,
              kBarVFree = 10, kBarSFull = 12, kBarPFull = 14, kBarODone = 16, kNumBars = 18;
constexpr uint32_t kTmemCols = 512;  // S0/P0, S1/P1, then O0, O1
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kTailStarts = 1, kHead = 2, kHeadEnds = 4;  // of a CTA, for the merge

template <int D>
struct Plan {
  static constexpr int NH = D / 64;
  static constexpr uint32_t kOffK = 2 * NH * kHalf;
  static constexpr uint32_t kOffV = 4 * NH * kHalf;
  static constexpr uint32_t kOffMl = 6 * NH * kHalf;               // [2][128] float2
  static constexpr uint32_t kOffBar = kOffMl + 2 * kRows * 8;
  static constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;     // TMEM base, abort, counts
  static constexpr uint32_t kOffPfx = (kOffMisc + 8 + 4 * kNumBars + 7) / 8 * 8;
  static constexpr size_t smem(int B) { return 1024 + kOffPfx + 8 * ((size_t)B + 1); }
};
static_assert(Plan<128>::smem(kTreeMaxBatch) <= 227 * 1024, "the largest batch fits");
template <bool B>
struct Masked {
  static constexpr bool value = B;
};

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
  float2* xml = reinterpret_cast<float2*>(base_ptr + PL::kOffMl);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(base_ptr + PL::kOffMisc);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(base_ptr + PL::kOffMisc + 4);
  volatile int32_t* armed = reinterpret_cast<volatile int32_t*>(base_ptr + PL::kOffMisc + 8);
  int64_t* pfx = reinterpret_cast<int64_t*>(base_ptr + PL::kOffPfx);  // [B+1] costs before

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
    pfx[b + 1] = tree_seq_cost(p.Hkv, n * G, tree_blocks(ctx));
  }
  __syncthreads();
  if (warp == 0) {
    int64_t carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int i = b0 + lane + 1;
      int64_t v = i <= p.B ? pfx[i] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += u;
      }
      if (i <= p.B) pfx[i] = v + carry;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t cost = pfx[p.B];
  const int64_t shares = tree_shares(cost, gridDim.x);
  const int64_t lo = blockIdx.x < shares ? tree_share(blockIdx.x, cost, shares) : 0;
  const int64_t hi = blockIdx.x < shares ? tree_share(blockIdx.x + 1, cost, shares) : 0;

  // Every role steps through the same parts.  Stream t's i-th block of a part is
  // j0 + i (two tiles) or j0 + 2 i + t (one), in buffer i & 1 or t; Q's tiles are in
  // slots 0 and 1 (two) or in one of them, in turn (one).  Use counts of buffers,
  // streams and slots run on from part to part (they give the barriers' phases).
  struct Walk {
    TreePart s;
    int q0, n, ctx;                                // rows of q, nodes, length
    int buf0 = 0, buf1 = 0, str0 = 0, str1 = 0;    // uses before this part
    int qu0 = 0, qu1 = 0, turn = 0;
    __device__ int count(int t) const { return s.two ? s.nblk : (s.nblk + 1 - t) / 2; }
    __device__ int block(int t, int i) const { return s.j0 + (s.two ? i : 2 * i + t); }
    __device__ int buf(int t, int i) const { return s.two ? i & 1 : t; }
    __device__ int use(int t, int i) const {
      return (buf(t, i) ? buf1 : buf0) + (s.two ? i >> 1 : i);
    }
    __device__ int str(int t) const { return t ? str1 : str0; }
    __device__ int slot(int t) const { return s.two ? t : turn; }
    __device__ int slot_use(int sl) const { return sl ? qu1 : qu0; }
    __device__ void done() {
      buf0 += (s.nblk + 1) / 2;
      buf1 += s.nblk / 2;
      str0 += count(0);
      str1 += count(1);
      if (s.two || turn == 0) ++qu0;
      if (s.two || turn == 1) ++qu1;
      if (!s.two) turn ^= 1;
    }
  } wk;
  int64_t at = lo;
  auto next = [&]() -> bool {
    while (at < hi) {
      int a = 0, z = p.B;  // the sequence holding `at`: the last with pfx <= at
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (pfx[mid] <= at) a = mid; else z = mid;
      }
      wk.s.b = a;
      seq_of(p, a, wk.q0, wk.n, wk.ctx);
      at += tree_part(p.Hkv, wk.n * G, tree_blocks(wk.ctx), at - pfx[a], hi - at, wk.s);
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

  if (warp >= 9) {
    const bool v = warp == 10;  // V, else Q and K: neither waits for the other's buffers
    // ------------------------------------------------------------ copies
    bool ok = true;
    while (ok && next()) {
      const int pages = (wk.ctx + kPageSize - 1) / kPageSize;
      const int32_t* table = p.block_tables + (int64_t)wk.s.b * p.MBS;
      const int streams = wk.s.two ? 1 : 2;
      auto entry = [&](int t, int i) -> int {  // lane l < 8: page l's block
        const int pg = wk.block(t, i) * kPages + lane;
        return lane < kPages && t < streams && i < wk.count(t) && pg < pages ? table[pg] : 0;
      };
      int cur0 = entry(0, 0), cur1 = entry(1, 0);
      for (int t = 0; ok && !v && t < (wk.s.two ? 2 : 1); ++t) {
        const int sl = wk.slot(t), u = wk.slot_use(sl);
        if (u > 0) ok = __all_sync(0xffffffffu, wait(kBarQFree + sl, (uint32_t)((u - 1) & 1)));
        if (!ok) break;
        if (lane == 0) {
          armed[kBarQ + sl] = armed[kBarQ + sl] + 1;
          mbar_arrive_expect_tx(bar(kBarQ + sl), NH * kHalf);
          for (int c = 0; c < NH; ++c)
            tma_load_3d(base + (uint32_t)(sl * NH + c) * kHalf, &tmq, bar(kBarQ + sl), c * 64,
                        wk.s.h * G, wk.q0 + (2 * wk.s.pair + t) * (kRows / G));
        }
      }
      for (int i = 0; ok && i < wk.count(0); ++i) {
        const int nxt0 = entry(0, i + 1), nxt1 = entry(1, i + 1);
        for (int t = 0; t < streams; ++t) {
          if (i >= wk.count(t)) continue;
          const int bb = wk.buf(t, i), u = wk.use(t, i);
          const int npg = min(kPages, pages - wk.block(t, i) * kPages);
          int blk = t == 0 ? cur0 : cur1;
          if (lane < npg && (blk < 0 || blk >= p.NB)) {  // zeros, past the pool
            if (!v) report_error(p.err_word, PKV_ERR_BOUNDS);
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
      // sl: Q's slot; bb: the buffer; last: nothing uses the buffer after this;
      // q_last: nothing uses the slot
      auto qk = [&](int t, int sl, int bb, bool last, bool q_last) {
        const uint64_t a0 = dq + (sl ? (uint64_t)NH * kHalf >> 4 : 0ull);
        const uint64_t b0 = dk + (bb ? (uint64_t)NH * kHalf >> 4 : 0ull);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (uint32_t)(ks >> 2) * kHalf + (uint32_t)(ks & 3) * 32;
          umma(tmem + (uint32_t)t * kTok, a0 + (off >> 4), b0 + (off >> 4), kIdS, ks > 0);
        }
        commit(kBarSFull + t);
        if (last) commit(kBarKFree + bb);
        if (q_last) commit(kBarQFree + sl);
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
      // The first product over O_t of a part comes after P_t, which the softmax
      // threads hand over after they have read the last part's accumulators out.
      while (ok && next()) {
        if (wk.s.two) {  // one buffer after the other, both streams from it
          const int n = wk.s.nblk;
          uint32_t u0 = (uint32_t)wk.buf0, u1 = (uint32_t)wk.buf1;  // uses of the next block's
          const uint32_t st = (uint32_t)wk.str0, st1 = (uint32_t)wk.str1;
          ok = wait(kBarKFull, u0 & 1) && wait(kBarQ, (uint32_t)wk.qu0 & 1);
          if (!ok) break;
          tc_fence_after();
          qk(0, 0, 0, false, n == 1);
          if (!(ok = wait(kBarQ + 1, (uint32_t)wk.qu1 & 1))) break;
          qk(1, 1, 0, true, n == 1);
          for (int i = 0; ok && i < n; ++i) {
            const int bb = i & 1;
            const bool more = i + 1 < n, end = i + 2 == n;
            const uint32_t vu = bb ? u1 : u0, ku = bb ? u0 + 1 : u1;  // this V, the next K
            if (!(ok = wait(kBarPFull, (st + i) & 1) && wait(kBarVFull + bb, vu & 1))) break;
            tc_fence_after();
            pv(0, bb, i > 0, false);
            if (more) {
              if (!(ok = wait(kBarKFull + (bb ^ 1), ku & 1))) break;
              qk(0, 0, bb ^ 1, false, end);
            }
            if (!(ok = wait(kBarPFull + 1, (st1 + i) & 1))) break;
            tc_fence_after();
            pv(1, bb, i > 0, true);
            if (more) qk(1, 1, bb ^ 1, true, end);
            if (bb) {
              ++u0;
              ++u1;
            }
          }
        } else {  // stream t from buffer t
          const int n0 = wk.count(0), n1 = wk.count(1), sl = wk.turn;
          const uint32_t u[2] = {(uint32_t)wk.buf0, (uint32_t)wk.buf1};
          const uint32_t st[2] = {(uint32_t)wk.str0, (uint32_t)wk.str1};
          // the last product with Q is stream 1's where both have as many blocks
          ok = wait(kBarQ + sl, (uint32_t)wk.slot_use(sl) & 1);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == 1 && n1 == 0) break;
            ok = ok && wait(kBarKFull + t, u[t] & 1);
            if (!ok) break;
            tc_fence_after();
            qk(t, sl, t, true, wk.s.nblk == 1 + t);
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
                qk(t, sl, t, true, 2 * (i + 1) + t == wk.s.nblk - 1);
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
    int flags = 0, tail_b = 0, tail_seg = 0;  // for the merge
    auto all_ok = [](bool mine) -> bool {  // both streams' 256 threads
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.and.pred q, 2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(r) : "r"((uint32_t)mine) : "memory");
      return r != 0;
    };
    bool ok = true;
    while (ok && next()) {
      const int nt = wk.count(t), done = wk.str(t);
      const int tok_step = wk.s.two ? kTok : 2 * kTok;
      int tok0 = wk.block(t, 0) * kTok;
      const int pages = (wk.ctx + kPageSize - 1) / kPageSize;
      const int32_t* table = p.block_tables + (int64_t)wk.s.b * p.MBS;
      const int row = (2 * wk.s.pair + (wk.s.two ? t : 0)) * kRows + tt;  // node x g + head
      const bool real = row < wk.n * G;
      const int past = wk.ctx - wk.n;
      // the nodes that the row sees, and those that any row of the tree does
      const uint64_t nodes = wk.n == 64 ? ~0ull : (1ull << wk.n) - 1;
      uint64_t mask = real ? (uint64_t)p.tree_mask[wk.q0 + row / G] & nodes : 0ull;
      uint64_t any = lane < wk.n ? (uint64_t)p.tree_mask[wk.q0 + lane] : 0ull;
      if (lane + 32 < wk.n) any |= (uint64_t)p.tree_mask[wk.q0 + lane + 32];
      any = ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32)) << 32 |
             __reduce_or_sync(0xffffffffu, (uint32_t)any)) & nodes;
      float m_ref = -INFINITY, l_sum = 0.f;
      for (int i = 0; i < nt; ++i, tok0 += tok_step) {
        // a block outside the pool (reported by the copy warp, zeros in shared
        // memory) is left out: bit pg stands for the step's page pg
        const int pg = tok0 / kPageSize + lane;
        const int entry = lane < kPages && pg < pages ? table[pg] : 0;
        ok = __all_sync(0xffffffffu, wait(kBarSFull + t, (uint32_t)((done + i) & 1)));
        if (!ok) break;
        tc_fence_after();
        const uint32_t bad = __ballot_sync(0xffffffffu, entry < 0 || entry >= p.NB);
        const bool full = tok0 + kTok <= past && bad == 0;
        // bit e: whether the row sees token tok0 + 32 qq + e
        auto sees = [&](int qq) -> uint32_t {
          const int s = tok0 + 32 * qq - past;  // of the tree's node 0, negative in the past
          uint32_t v = s <= -32 ? 0xffffffffu : s >= 64 ? 0u : s >= 0 ? (uint32_t)(mask >> s)
                       : (uint32_t)(mask << -s) | ((1u << -s) - 1);
          if ((bad >> (2 * qq)) & 1) v &= 0xffff0000u;
          if ((bad >> (2 * qq + 1)) & 1) v &= 0x0000ffffu;
          return v;
        };
        uint32_t sa[32], sb[32];
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto qmax = [&](auto mc, const uint32_t (&sq)[32], int qq) {
          [[maybe_unused]] uint32_t v = 0;
          if constexpr (decltype(mc)::value) v = sees(qq);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a = __uint_as_float(sq[2 * e]), c = __uint_as_float(sq[2 * e + 1]);
            if constexpr (decltype(mc)::value) {
              if (!(v & (1u << (2 * e)))) a = -INFINITY;
              if (!(v & (2u << (2 * e)))) c = -INFINITY;
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
        auto qp = [&](auto mc, const uint32_t (&sq)[32], int qq) {
          [[maybe_unused]] uint32_t v = 0;
          if constexpr (decltype(mc)::value) v = sees(qq);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = f2_split(fma2(f2(__uint_as_float(sq[2 * e]),
                                              __uint_as_float(sq[2 * e + 1])), c2x2, nmu2));
            float p0 = ex2(y.x), p1 = ex2(y.y);
            if constexpr (decltype(mc)::value) {
              if (!(v & (1u << (2 * e)))) p0 = 0.f;
              if (!(v & (2u << (2 * e)))) p1 = 0.f;
            }
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
        // V rows behind the end, and of nodes that no row sees, may hold anything
        // (0 x NaN): zeroed in the staged block by the stream that uses it first
        if (tok0 + kTok > past && (t == 0 || !wk.s.two)) {
          const int bb = wk.buf(t, i);
          ok = __all_sync(0xffffffffu, wait(kBarVFull + bb, (uint32_t)(wk.use(t, i) & 1)));
          if (!ok) break;
          const int first = max(0, past - tok0);
          const uint32_t vb = base + kOffV + (uint32_t)bb * NH * kHalf;
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
      // ---- the part's end: both accumulators of one tile join
      const int nt1 = wk.count(t ^ 1), done1 = wk.str(t ^ 1);
      const bool join = !wk.s.two && nt1 > 0 && nt > 0;  // two streams, one tile
      if (ok && nt > 0)
        ok = __all_sync(0xffffffffu, wait(kBarODone + t, (uint32_t)((done + nt - 1) & 1)));
      if (ok && join)
        ok = __all_sync(0xffffffffu, wait(kBarODone + (t ^ 1), (uint32_t)((done1 + nt1 - 1) & 1)));
      float a_me = 1.f, a_it = 0.f;
      if (join) {  // (also where a wait gave up: both streams take part)
        xml[t * kRows + tt] = make_float2(m_ref, l_sum);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float2 o = xml[(t ^ 1) * kRows + tt];
        const float M = fmaxf(m_ref, o.x);
        const float mu = M == -INFINITY ? 0.f : M;
        a_me = ex2(m_ref - mu);
        a_it = ex2(o.x - mu);
        // the same sum in both streams
        const float la = t == 0 ? a_me * l_sum : a_it * o.y, lb = t == 0 ? a_it * o.y : a_me * l_sum;
        l_sum = la + lb;
        m_ref = M;
      }
      if (ok && nt > 0) {
        tc_fence_after();
        const bool head = wk.s.j0 > 0, ends = wk.s.j0 + wk.s.nblk == wk.s.total;
        const bool whole = !head && ends;
        const bool some = l_sum != 0.f;  // NaN counts: it has to show
        const int64_t prow = (2 * (int64_t)blockIdx.x + (head ? 0 : 1)) * (2 * kRows) +
                             (wk.s.two ? t * kRows : 0) + tt;
        const float inv = some ? 1.f / l_sum : 0.f;
        const int64_t orow = (int64_t)(wk.q0 + row / G) * p.Hq + wk.s.h * G + row % G;
        if (!whole) {
          if (head) flags |= kHead | (ends ? kHeadEnds : 0);
          else {
            flags |= kTailStarts;
            tail_b = wk.s.b;
            tail_seg = wk.s.pair * p.Hkv + wk.s.h;
          }
          if (real && (t == 0 || !join))
            p.part_ml[prow] = some ? make_float2(m_ref, l_sum) : make_float2(-INFINITY, 0.f);
        }
        const uint32_t t_it = tmem + 256 + (uint32_t)(t ^ 1) * D + lane_base;
        const int c_lo = join && t == 1 ? D / 64 : 0, c_hi = join && t == 0 ? D / 64 : D / 32;
#pragma unroll 1
        for (int cc = c_lo; cc < c_hi; ++cc) {
          uint32_t r[32], r2[32];
          tmem_ld32(t_o + (uint32_t)cc * 32, r);
          if (join) {
            tmem_ld32(t_it + (uint32_t)cc * 32, r2);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              // stream 0's share first, whichever thread adds
              const float mine = a_me * __uint_as_float(r[e]), its = a_it * __uint_as_float(r2[e]);
              r[e] = __float_as_uint(mine + its);
            }
          }
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
        tc_fence_before();  // the accumulators are read before P_t of the next part
      }
      // neither stream's next part touches an accumulator the other still reads,
      // nor the exchanged (m, l); and both go on, or neither
      ok = all_ok(ok);
      wk.done();
    }
    if (tid == 0) p.meta[blockIdx.x] = make_int4(flags, tail_b, tail_seg, 0);
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

// ---- the merge of the segments that share boundaries cut: a warp per row
constexpr int kMergeWarps = 4;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const TreeParams p) {
  constexpr int V = D / 32;  // columns per lane
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, c = blockIdx.x;
  const int r = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);  // row of the pair
  const int4 mt = p.meta[c];
  if (!(mt.x & kTailStarts)) return;
  const int G = p.Hq / p.Hkv, b = mt.y, pair = mt.z / p.Hkv, h = mt.z - pair * p.Hkv;
  int q0, n, ctx;
  if (!seq_of(p, b, q0, n, ctx)) return;
  const int row = pair * 2 * kRows + r;
  if (row >= n * G) return;
  // the parts: slot 2 c + 1, then 2 c' of the CTAs behind, up to the one whose
  // part ends the segment
  int last = c + 1;
  while (last < p.ctas - 1 && !(p.meta[last].x & kHeadEnds)) ++last;
  const int parts = last - c + 1;
  auto slot = [&](int k) -> int64_t {
    return (k == 0 ? 2 * (int64_t)c + 1 : 2 * (int64_t)(c + k)) * (2 * kRows) + r;
  };
  float M = -INFINITY;
  for (int k = lane; k < parts; k += 32) M = fmaxf(M, p.part_ml[slot(k)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (M == -INFINITY) M = 0.f;  // nothing at all, or nothing but NaN
  float acc[V] = {}, l = 0.f;
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const int64_t s = slot(k);
    const float2 ml = p.part_ml[s];
    if (ml.y == 0.f) continue;  // a part with nothing in it
    const float w = ex2(ml.x - M);
    l += w * ml.y;
    const float* x = p.part_o + s * D + lane * V;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] += w * x[e];
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const int64_t to = ((int64_t)(q0 + row / G) * p.Hq + h * G + row % G) * D + lane * V;
  if (p.out_dtype == PKV_F32) {
#pragma unroll
    for (int e = 0; e < V; ++e) static_cast<float*>(p.out)[to + e] = acc[e] * inv;
  } else {
    const bool bf = p.out_dtype == PKV_BF16;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + to);
#pragma unroll
    for (int e = 0; e < V / 2; ++e)
      out[e] = bf ? pack2<true>(acc[2 * e] * inv, acc[2 * e + 1] * inv)
                  : pack2<false>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
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
  if (e != cudaSuccess || l.p.ctas < 2) return e;
  int rows = l.p.max_q * (l.p.Hq / l.p.Hkv);
  if (rows > 2 * kRows) rows = 2 * kRows;
  return launch_dependent(tree_merge_kernel<D>,
                          dim3((unsigned)l.p.ctas, (unsigned)((rows + kMergeWarps - 1) / kMergeWarps)),
                          dim3(kMergeWarps * 32), 0, l.stream, l.p);
}

}  // namespace tr

cudaError_t launch_tree(const TreeLaunch& l) {
  if (l.d == 64) return l.bf16 ? tr::launch<true, 64>(l) : tr::launch<false, 64>(l);
  if (l.d == 128) return l.bf16 ? tr::launch<true, 128>(l) : tr::launch<false, 128>(l);
  return cudaErrorNotSupported;
}

}  // namespace pkv
