// Paged prefill attention with the scores changed before the softmax: capped by
// a tanh, given a bias that grows with the distance, or both.
//
// The work of the prefill kernel (pkv_prefill.cu): one CTA per 256 query rows,
// 256 / g new tokens of one sequence times the g query heads of one KV head, in
// two tiles of 128 rows; warps 0-3 and 4-7 run the softmax of tile 0 and 1 (one
// row per thread, TMEM lane t), warp 8 issues the MMAs, warp 9 the copies.  A
// cap costs an exponential and a reciprocal per score, which makes the softmax
// the longer part, so the pipeline differs: N steps of 64 cached tokens, per step
// and tile
//   S = Q K^T   tcgen05.mma M 128 x N 64 x K d, from shared memory;
//   softmax     the row's 64 scores are read once, P goes back over them as hi +
//               lo 16-bit pairs (the weights keep about 16 bits);
//   O += P V    tcgen05.mma with A from tensor memory, twice per 16 tokens.
// Tensor memory holds two S / P buffers of 64 columns per tile beside the two
// accumulators (512 columns at d 128), so the scores of step i + 1 are there
// when the softmax of step i ends: a tile's softmax runs without a break, and
// waits for its products only to rescale O, which it seldom does.
// Four sequences of 2048 rows behind 6144 tokens, 32/8 heads of 128, capped:
// 1399 us, against 1488 with the prefill kernel's steps of 128 tokens and one
// buffer, where a tile's softmax and its products take turns; 1370 with the MMAs
// issued behind elect.sync.  12 sequences of up to 700 rows with cap and slopes:
// 189, before 208.  A step takes about 3500 cycles.  No pipe is full in the long
// case (tensor 45 %, special functions 46 %, issue 45 %): what is left is the
// latency of the two softmax warps of a scheduler.  Twice the warps, two groups per
// tile that take the steps in turn and hand the reference maximum over, took
// 1482 us (96 registers).
#pragma once

#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace pfb {

constexpr int kRows = 128, kTok = 64, kPages = kTok / kPageSize, kSlots = 4;
constexpr int kThreads = 320;
constexpr uint32_t kQHalf = 16384;   // 128 rows x 128 bytes: 64 d columns of a Q tile
constexpr uint32_t kSHalf = 8192;    // 64 rows x 128 bytes: the same of a K or V step
constexpr int kBarQ = 0, kBarKFull = 1, kBarVFull = 5, kBarKFree = 9, kBarVFree = 13,
              kBarSFull = 17, kBarPFull = 21, kBarODone = 25, kBarDrain = 29, kNumBars = 30;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 1000000000ull;

template <int D>
struct Plan {
  static constexpr int NH = D / 64;
  static constexpr uint32_t kOffK = 2 * NH * kQHalf;
  static constexpr uint32_t kOffV = kOffK + kSlots * NH * kSHalf;
  static constexpr uint32_t kOffBar = kOffV + kSlots * NH * kSHalf;
  static constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;  // TMEM base, abort, counts
  static constexpr size_t kSmem = 1024 + kOffMisc + 8 + 4 * kNumBars;
  static_assert(D == 64 || D == 128, "head dims built");
};
template <bool B>
struct Masked {
  static constexpr bool value = B;
};

// A CTA's shared memory, tensor memory and flags.
struct Cta {
  uint32_t base, tmem;
  uint8_t* ptr;
  volatile int32_t* abort_flag;
  volatile int32_t* armed;  // copies armed on each barrier
  uint32_t off_bar;
  __device__ uint32_t bar(int i) const { return base + off_bar + 8u * (uint32_t)i; }
  // A bounded wait; one that gives up raises the CTA's abort flag, after which
  // no role waits any more.
  __device__ bool wait(int i, uint32_t parity) const {
    if (mbar_try_wait(bar(i), parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait_bounded(bar(i), parity, kWaitNs)) return true;
    *abort_flag = 1;
    return false;
  }
  __device__ bool wait_warp(int i, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait(i, parity));
  }
};

// All threads, before the first role: barriers and tensor memory.
template <int D>
__device__ __forceinline__ Cta setup(uint8_t* smem_raw) {
  using PL = Plan<D>;
  const uint32_t raw = smem_u32(smem_raw);
  Cta c;
  c.base = (raw + 1023u) & ~1023u;
  c.ptr = smem_raw + (c.base - raw);
  c.off_bar = PL::kOffBar;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(c.ptr + PL::kOffMisc);
  c.abort_flag = reinterpret_cast<volatile int32_t*>(c.ptr + PL::kOffMisc + 4);
  c.armed = reinterpret_cast<volatile int32_t*>(c.ptr + PL::kOffMisc + 8);
  if (threadIdx.x < 32) {
    tmem_alloc(c.base + PL::kOffMisc, kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    *c.abort_flag = 0;
    for (int i = 0; i < kNumBars; ++i) {
      c.armed[i] = 0;
      mbar_init(c.bar(i), i >= kBarPFull && i < kBarODone ? kRows / 32 : 1);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  c.tmem = *slot;
  return c;
}
// All threads, after the last role.
__device__ __forceinline__ void teardown(const Cta& c, int32_t* err_word) {
  tc_fence_before();
  __syncthreads();
  if (*c.abort_flag) {  // let copies and MMAs in flight land before the memory is given back
    const int i = threadIdx.x;
    if (i == 0) report_error(err_word, PKV_ERR_TIMEOUT);
    if (i < kBarKFree && c.armed[i] > 0)
      mbar_wait_bounded(c.bar(i), (uint32_t)((c.armed[i] - 1) & 1), kWaitNs);
    if (i >> 5 == 8 && elect_one()) {  // the thread that issued the MMAs
      umma_commit(c.bar(kBarDrain));
      mbar_wait_bounded(c.bar(kBarDrain), 0, kWaitNs);
    }
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    tc_fence_after();
    tmem_dealloc(c.tmem, kTmemCols);
  }
}

// The copy warp: the N steps of the blocks in `table`, of which `pages` pages
// exist.  A block outside the pool is reported and read as zeros (past the pool's
// end).
template <int D>
__device__ __forceinline__ void copy_steps(const Cta& c, int N, const void* tmk, const void* tmv,
                                           const int32_t* table, int pages, int h, int Hkv, int NB,
                                           int32_t* err_word) {
  using PL = Plan<D>;
  constexpr int NH = PL::NH;
  const int lane = threadIdx.x & 31;
  // lane l holds page 32 g + l, the next 32 looked up one group ahead
  const int end = min(pages, N * kPages);
  auto look_up = [&](int g) -> int {
    const int pg = 32 * g + lane;
    return pg < end ? table[pg] : 0;
  };
  int cur = 0, nxt = look_up(0);
  for (int x = 0; x < N; ++x) {
    if ((x & 7) == 0) {
      cur = nxt;
      nxt = look_up((x >> 3) + 1);
    }
    const int npg = min(kPages, pages - x * kPages);
    int blk = __shfl_sync(0xffffffffu, cur, ((x & 7) * kPages + lane) & 31);
    if (lane < npg && (blk < 0 || blk >= NB)) {
      report_error(err_word, PKV_ERR_BOUNDS);
      blk = NB;
    }
    const uint32_t s = (uint32_t)x & (kSlots - 1), u = (uint32_t)x / kSlots;
    for (int v = 0; v < 2; ++v) {
      const int full = (v ? kBarVFull : kBarKFull) + (int)s;
      if (u > 0 && !c.wait_warp((v ? kBarVFree : kBarKFree) + (int)s, (u - 1) & 1)) return;
      if (lane == 0) {
        c.armed[full] = c.armed[full] + 1;
        mbar_arrive_expect_tx(c.bar(full), (uint32_t)npg * NH * kPageSize * 128);
      }
      __syncwarp();
      if (lane < npg) {
        const uint32_t dst = c.base + (v ? PL::kOffV : PL::kOffK) + s * NH * kSHalf +
                             (uint32_t)lane * kPageSize * 128;
        const int row = (blk * Hkv + h) * kPageSize;
        for (int k = 0; k < NH; ++k)
          tma_load_2d_plain(dst + (uint32_t)k * kSHalf, v ? tmv : tmk, c.bar(full), k * 64, row);
      }
    }
    if (__any_sync(0xffffffffu, *c.abort_flag != 0)) return;
  }
}

// The MMA warp's elected lane.
template <bool BF16, int D>
__device__ __forceinline__ void mma_steps(const Cta& c, int N) {
  using PL = Plan<D>;
  constexpr int NH = PL::NH;
  constexpr uint32_t kIdS = idesc_f16(BF16, false, kRows, kTok);
  constexpr uint32_t kIdO = idesc_f16(BF16, true, kRows, D);
  const uint64_t dq = sdesc(c.base, 16, 1024);
  const uint64_t dk = sdesc(c.base + PL::kOffK, 16, 1024);
  const uint64_t dv = sdesc(c.base + PL::kOffV, kSHalf, 1024);
  auto qk = [&](int t, int i) -> bool {  // scores of tile t's step i
    const uint32_t s = (uint32_t)i & (kSlots - 1), sb = (uint32_t)i & 1;
    if (t == 0) {
      if (!c.wait(kBarKFull + (int)s, ((uint32_t)i / kSlots) & 1)) return false;
      tc_fence_after();
    }
    const uint64_t a0 = dq + (t ? (uint64_t)NH * kQHalf >> 4 : 0ull);
    const uint64_t b0 = dk + ((uint64_t)s * NH * kSHalf >> 4);
    const uint32_t d0 = c.tmem + (uint32_t)t * 128 + sb * kTok;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint32_t in = (uint32_t)(ks & 3) * 32;
      umma(d0, a0 + (((uint32_t)(ks >> 2) * kQHalf + in) >> 4),
           b0 + (((uint32_t)(ks >> 2) * kSHalf + in) >> 4), kIdS, ks > 0);
    }
    umma_commit(c.bar(kBarSFull + 2 * t + (int)sb));
    if (t == 1) umma_commit(c.bar(kBarKFree + (int)s));
    return true;
  };
  auto pv = [&](int t, int i) -> bool {
    const uint32_t s = (uint32_t)i & (kSlots - 1), sb = (uint32_t)i & 1;
    if (!c.wait(kBarPFull + 2 * t + (int)sb, ((uint32_t)i >> 1) & 1)) return false;
    if (t == 0 && !c.wait(kBarVFull + (int)s, ((uint32_t)i / kSlots) & 1)) return false;
    tc_fence_after();
    const uint64_t b0 = dv + ((uint64_t)s * NH * kSHalf >> 4);
    const uint32_t pt = c.tmem + (uint32_t)t * 128 + sb * kTok;  // 32 columns of hi, 32 of lo
    const uint32_t dt = c.tmem + 256 + (uint32_t)t * D;
#pragma unroll
    for (int ks = 0; ks < kTok / 16; ++ks) {
      const uint64_t bv = b0 + ((uint32_t)ks * 16 * 128 >> 4);
      umma_ts(dt, pt + (uint32_t)ks * 8, bv, kIdO, i > 0 || ks > 0);
      umma_ts(dt, pt + 32 + (uint32_t)ks * 8, bv, kIdO, 1);
    }
    umma_commit(c.bar(kBarODone + 2 * t + (int)sb));
    if (t == 1) umma_commit(c.bar(kBarVFree + (int)s));
    return true;
  };
  if (!c.wait(kBarQ, 0)) return;
  for (int i = 0; i < min(N, 2); ++i) {
    if (!qk(0, i) || !qk(1, i)) return;
  }
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (!pv(t, i)) return;
      // the scores two steps on take the buffer that P leaves (MMAs of one thread
      // run in issue order)
      if (i + 2 < N && !qk(t, i + 2)) return;
    }
  }
}

// What is done to the scores, and what a row sees.
struct Row {
  float c2;                // scale log2e
  int vis;                 // last position the row sees
  int all_vis;             // last position every row of the warp sees
  int v_end;               // V rows from this position on may hold anything
  float cap_log2, cap_z;   // see cap_score
  float slope2;            // distance slope, log2 units
};

// The softmax warps of tile t: row tt (0 .. 127).  Leaves the row's sum; its O is
// complete in tensor memory when this returns true.
template <bool BF16, int D, int BIAS>
__device__ __forceinline__ bool softmax_steps(const Cta& c, int N, int t, int tt, const Row& w,
                                              float& l_sum) {
  using PL = Plan<D>;
  constexpr int NH = PL::NH;
  constexpr bool kCap = (BIAS & kBiasCap) != 0, kDist = (BIAS & kBiasDist) != 0;
  static_assert(kCap || kDist, "plain scores: pkv_prefill.cu");
  const int lane = threadIdx.x & 31;
  const uint32_t lane_base = (uint32_t)(tt & ~31) << 16;
  const uint32_t t_o = c.tmem + 256 + (uint32_t)t * D + lane_base;
  const uint64_t c2x2 = f2(w.c2, w.c2);
  const uint64_t cz2 = f2(w.cap_z, w.cap_z), cap2 = f2(w.cap_log2, w.cap_log2),
                 mcap2 = f2(-2.f * w.cap_log2, -2.f * w.cap_log2);
  const uint64_t dist_step = f2(2.f * w.slope2, 2.f * w.slope2);
  // two raw scores capped, plus `add`, which holds the cap: see cap_score
  auto cap_pair = [&](uint64_t raw, uint64_t add) -> uint64_t {
    const float2 z = f2_split(mul2(raw, cz2));
    const float2 u = f2_split(add2(f2(ex2(z.x), ex2(z.y)), f2(1.f, 1.f)));
    return fma2(f2(rcp(u.x), rcp(u.y)), mcap2, add);
  };
  float m_ref = -INFINITY;
  l_sum = 0.f;
  for (int i = 0; i < N; ++i) {
    const int tok0 = i * kTok;
    const uint32_t sb = (uint32_t)i & 1;
    const uint32_t t_s = c.tmem + (uint32_t)t * 128 + sb * kTok + lane_base;
    if (!c.wait_warp(kBarSFull + 2 * t + (int)sb, ((uint32_t)i >> 1) & 1)) return false;
    tc_fence_after();
    const bool full = tok0 + kTok - 1 <= w.all_vis;  // no row masks anything here
    uint32_t a[2][32];
    tmem_ld32_issue(t_s, a[0]);
    tmem_ld32_issue(t_s + 32, a[1]);
    tmem_ld_wait(a[0]);
    tmem_ld_wait(a[1]);
    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    auto max_pass = [&](auto mc) {
#pragma unroll
      for (int qq = 0; qq < 2; ++qq) {
        const int t0 = tok0 + 32 * qq;
        // the distance bias of two tokens, and the cap; stepped on by adding, so the
        // last of 32 tokens carries 16 roundings of its bias where a product for each
        // would carry one
        [[maybe_unused]] uint64_t add = f2(w.slope2 * (float)(t0 - w.vis),
                                           w.slope2 * (float)(t0 + 1 - w.vis));
        if constexpr (kCap) add = add2(cap2, add);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 v = make_float2(__uint_as_float(a[qq][2 * e]), __uint_as_float(a[qq][2 * e + 1]));
          if constexpr (kDist) {  // changed here, in place, for the P pass
            if constexpr (kCap) v = f2_split(cap_pair(f2(v.x, v.y), add));
            else v = f2_split(fma2(f2(v.x, v.y), c2x2, add));
            add = add2(add, dist_step);
          }
          if constexpr (decltype(mc)::value) {
            if (t0 + 2 * e > w.vis) v.x = -INFINITY;
            if (t0 + 2 * e + 1 > w.vis) v.y = -INFINITY;
          }
          m4[e & 3] = max3(m4[e & 3], v.x, v.y);
          if constexpr (kDist) {
            a[qq][2 * e] = __float_as_uint(v.x);
            a[qq][2 * e + 1] = __float_as_uint(v.y);
          }
        }
      }
    };
    if (full) max_pass(Masked<false>{});
    else max_pass(Masked<true>{});
    float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
    if constexpr (!kDist) {  // a cap alone keeps the order of the scores: the largest alone
      if (mx > -INFINITY) mx = f2_split(cap_pair(f2(mx, mx), cap2)).x;
    }
    // lazy rescale: keep the reference max while scores stay within 2^8 of it
    const bool grow = mx > m_ref + 8.f;
    float alpha = 1.f;
    if (grow) {
      alpha = ex2(m_ref - mx);  // 0 on the first step
      m_ref = mx;
      l_sum *= alpha;
    }
    if (i > 0 && __any_sync(0xffffffffu, grow)) {
      // O holds the steps before this one when P.V of the last is done.  Its barrier
      // alternates: most phases are never waited for, and a parity tells two
      // phases of one barrier apart only if the one before is known to be over,
      // here that of the step three back, issued before the last step's scores.
      if (!c.wait_warp(kBarODone + 2 * t + (int)(sb ^ 1), ((uint32_t)(i - 1) >> 1) & 1))
        return false;
      tc_fence_after();
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        tmem_ld32(t_o + (uint32_t)cc * 32, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
        tmem_st32(t_o + (uint32_t)cc * 32, o);
      }
    }
    const float mu = m_ref == -INFINITY ? 0.f : m_ref;
    const uint64_t sub = kCap && !kDist ? add2(cap2, f2(-mu, -mu)) : f2(-mu, -mu);
    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
    auto p_pass = [&](auto mc) {  // hi pairs over the first 32 columns, lo over the others
#pragma unroll
      for (int qq = 0; qq < 2; ++qq) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t raw = f2(__uint_as_float(a[qq][2 * e]), __uint_as_float(a[qq][2 * e + 1]));
          float2 v;
          if constexpr (kDist) v = f2_split(add2(raw, sub));
          else v = f2_split(cap_pair(raw, sub));
          float p0 = ex2(v.x), p1 = ex2(v.y);
          if constexpr (decltype(mc)::value && !kDist) {
            const int tk = tok0 + 32 * qq + 2 * e;
            if (tk > w.vis) p0 = 0.f;
            if (tk + 1 > w.vis) p1 = 0.f;
          }
          const uint64_t pp = f2(p0, p1);
          acc[e & 3] = add2(acc[e & 3], pp);
          hi[e] = pack2<BF16>(p0, p1);
          const float2 hf = unpack2<BF16>(hi[e]);
          const float2 l = f2_split(sub2(pp, f2(hf.x, hf.y)));
          lo[e] = pack2<BF16>(l.x, l.y);
        }
        tmem_st16_issue(t_s + 16u * qq, hi);
        tmem_st16_issue(t_s + 32u + 16u * qq, lo);
      }
    };
    if (full) p_pass(Masked<false>{});
    else p_pass(Masked<true>{});
    {
      const float2 a0 = f2_split(add2(acc[0], acc[1])), a1 = f2_split(add2(acc[2], acc[3]));
      l_sum += (a0.x + a0.y) + (a1.x + a1.y);
    }
    // V rows behind the context may hold anything (0 x NaN): zeroed in the staged
    // step by the tile that uses it first
    if (tok0 + kTok > w.v_end && t == 0) {
      const uint32_t s = (uint32_t)i & (kSlots - 1);
      if (!c.wait_warp(kBarVFull + (int)s, ((uint32_t)i / kSlots) & 1)) return false;
      const int from = max(0, w.v_end - tok0);
      const uint32_t vb = c.base + PL::kOffV + s * NH * kSHalf;
      for (int e = tt; e < (kTok - from) * 8 * NH; e += kRows) {
        const int rr = from + e / (8 * NH), ch = e % (8 * NH);
        const uint32_t ad = vb + (uint32_t)(ch >> 3) * kSHalf + (uint32_t)rr * 128 +
                            (uint32_t)(ch & 7) * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(ad), "r"(0) : "memory");
      }
      // the tensor cores read them through the async proxy
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar(kBarPFull + 2 * t + (int)sb));
  }
  if (!c.wait_warp(kBarODone + 2 * t + ((N - 1) & 1), ((uint32_t)(N - 1) >> 1) & 1)) return false;
  tc_fence_after();
  return true;
}

template <bool BF16, int D, int BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_biased_kernel(const PrefillParams p, const __grid_constant__ CUtensorMap tmq,
                          const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv) {
  using PL = Plan<D>;
  constexpr int NH = PL::NH;
  // the last rows of every sequence and head start first: they see the longest
  // stretch, and the short ones fill the end of the run
  const int rest = blockIdx.x / p.Hkv;
  const int h = blockIdx.x - rest * p.Hkv;                    // KV head
  const int ctile = p.tiles_per_seq - 1 - rest / p.B;         // pair of tiles
  const int b = rest - rest / p.B * p.B;                      // sequence
  const int G = p.Hq / p.Hkv;                                 // query heads per KV head
  const int tpt = kRows / G;                            // tokens per tile
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, and known to be

  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int q0 = p.q_start[b], qn = p.q_start[b + 1] - q0;    // this sequence's rows
  const int ctx = p.context_lens[b];
  if (qn < 0 || ctx < qn || ctx > p.MBS * kPageSize || q0 < 0 || q0 + qn > p.total_q ||
      qn > p.tiles_per_seq * 2 * tpt) {
    if (tid == 0 && ctile == 0 && h == 0) report_error(p.err_word, PKV_ERR_BOUNDS);
    return;
  }
  const int tok_base = ctile * 2 * tpt;  // first new token of the CTA
  if (tok_base >= qn) return;            // no rows of this sequence here

  extern __shared__ uint8_t smem_raw[];
  const Cta c = setup<D>(smem_raw);
  const int last_tok = min(qn, tok_base + 2 * tpt) - 1;
  const int N = (ctx - qn + last_tok) / kTok + 1;  // causal: steps any row sees

  if (warp == 9) {
    if (lane == 0) {
      prefetch_tmap(&tmq);
      prefetch_tmap(&tmk);
      prefetch_tmap(&tmv);
      c.armed[kBarQ] = 1;
      mbar_arrive_expect_tx(c.bar(kBarQ), 2 * NH * kQHalf);
      for (int t = 0; t < 2; ++t)
        for (int k = 0; k < NH; ++k)
          tma_load_3d(c.base + (uint32_t)(t * NH + k) * kQHalf, &tmq, c.bar(kBarQ),
                      k * 64, h * G, q0 + tok_base + t * tpt);
    }
    copy_steps<D>(c, N, &tmk, &tmv, p.block_tables + (int64_t)b * p.MBS,
                  (ctx + kPageSize - 1) / kPageSize, h, p.Hkv, p.NB, p.err_word);
  } else if (warp == 8) {
    if (elect_one()) mma_steps<BF16, D>(c, N);
  } else {
    const int t = warp >> 2, tt = tid - t * kRows;
    const int row = tok_base + t * tpt + tt / G;  // new token of this row
    const int hq = h * G + tt % G;
    Row w;
    w.c2 = p.scale_log2;
    w.vis = min(ctx - qn + row, ctx - 1);
    w.all_vis = min(ctx - qn + tok_base + t * tpt, ctx - 1);
    w.v_end = ctx;
    w.cap_log2 = p.cap_log2;
    w.cap_z = p.cap_z;
    w.slope2 = (BIAS & kBiasDist) != 0 ? p.slopes[hq] * 1.4426950408889634f : 0.f;
    float l_sum;
    if (softmax_steps<BF16, D, BIAS>(c, N, t, tt, w, l_sum)) {
      // ---- out = O / l for the tile's real rows
      const float inv = l_sum > 0.f ? 1.f / l_sum : 0.f;
      const uint32_t t_o = c.tmem + 256 + (uint32_t)t * D + ((uint32_t)(tt & ~31) << 16);
      const int64_t orow = ((int64_t)(q0 + row) * p.Hq + hq) * D;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        tmem_ld32(t_o + (uint32_t)cc * 32, o);
        if (row < qn) {
          if (p.out_dtype == PKV_F32) {
            float4* o4 = reinterpret_cast<float4*>(static_cast<float*>(p.out) + orow + cc * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o4[e] = make_float4(__uint_as_float(o[4 * e]) * inv,
                                  __uint_as_float(o[4 * e + 1]) * inv,
                                  __uint_as_float(o[4 * e + 2]) * inv,
                                  __uint_as_float(o[4 * e + 3]) * inv);
          } else {
            uint4* o4 = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + orow + cc * 32);
            const bool obf = p.out_dtype == PKV_BF16;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float x = __uint_as_float(o[8 * e + 2 * k]) * inv;
                const float y = __uint_as_float(o[8 * e + 2 * k + 1]) * inv;
                u[k] = obf ? pack2<true>(x, y) : pack2<false>(x, y);
              }
              o4[e] = make_uint4(u[0], u[1], u[2], u[3]);
            }
          }
        }
      }
    }
  }
  teardown(c, p.err_word);
}

template <bool BF16, int D, int BIAS>
cudaError_t launch_kernel(const PrefillLaunch& l) {
  auto kern = prefill_biased_kernel<BF16, D, BIAS>;
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
  const int64_t grid = (int64_t)l.p.B * l.p.tiles_per_seq * l.p.Hkv;
  if (grid >= (int64_t)1 << 31) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
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

template <int BIAS>
cudaError_t launch_bias(const PrefillLaunch& l) {
  if (l.d == 64)
    return l.bf16 ? launch_kernel<true, 64, BIAS>(l) : launch_kernel<false, 64, BIAS>(l);
  if (l.d == 128)
    return l.bf16 ? launch_kernel<true, 128, BIAS>(l) : launch_kernel<false, 128, BIAS>(l);
  return cudaErrorNotSupported;
}

}  // namespace pfb
}  // namespace pkv
