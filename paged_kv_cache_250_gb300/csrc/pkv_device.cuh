// pkv_device.cuh -- device-side building blocks for sm_103a: mbarriers, TMA
// tile loads, warp-level tensor-core fragments and the error word.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pkv.h"
#include "pkv_hd.h"

namespace pkv {

// ---------------------------------------------------------------- errors
// First device-detected error wins; later ones are dropped.
__device__ __forceinline__ void report_error(int32_t* err_word, int32_t code) {
  if (err_word != nullptr) atomicCAS(err_word, 0, code);
}

// ---------------------------------------------------------------- kernels in a row
// Wait for the kernel in front, then let the next one start its prologue.  In this
// order whatever starts behind finds all kernels but the last complete: a step may
// read lengths that an earlier kernel wrote while the one in front still runs
// (PKV_STEP_OVERLAP).
__device__ __forceinline__ void griddep_wait_then_trigger() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------- smem addr
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------- mbarrier
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count)
               : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait: gives up after roughly `limit_ns` nanoseconds of global-timer
// time and returns false.  Each try_wait already suspends the thread for a
// hardware-chosen interval, so the loop does not hammer the barrier.
__device__ __forceinline__ bool mbar_wait_bounded(uint32_t bar, uint32_t parity,
                                                  uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t1;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t1));
    if (t1 - t0 > limit_ns) return false;
  }
}

// ---------------------------------------------------------------- TMA
// 2-D tiled bulk tensor load global -> shared, completing on an mbarrier.
// x is the element column (must be a multiple of 16 bytes / element size),
// y the row.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, uint32_t bar,
                                            int32_t x, int32_t y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(tmap), "r"(bar), "r"(x), "r"(y), "l"(policy)
      : "memory");
}

// 1-D bulk copy global -> shared of `bytes` (a multiple of 16; both addresses
// 16-byte aligned), completing on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ uint64_t l2_policy_evict_first() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// Pull `bytes` (a multiple of 16, 16-byte aligned) at `src` into L2; no data
// changes hands and nothing waits for it.
__device__ __forceinline__ void l2_prefetch_bulk(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void prefetch_tmap(const void* tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(tmap) : "memory");
}

// ---------------------------------------------------------------- fragments
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ uint32_t movm_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// D = A * B + D, m16n8k16, fp32 accumulate.  IsBF16 selects bf16 operands,
// otherwise fp16.
template <bool IsBF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4],
                                          uint32_t b0, uint32_t b1) {
  if constexpr (IsBF16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// ---------------------------------------------------------------- scores
__device__ __forceinline__ float ex2(float x) {  // 2^x (PTX ex2.approx; -inf gives 0)
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {  // 1 / x (PTX rcp.approx; inf gives 0)
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A score x capped by a tanh, both in log2 units: with y = s / cap and
// z = 2 y log2e = x z_of_x (z_of_x = 2 / cap),  tanh(y) = 1 - 2 / (1 + 2^z):
// two special-function instructions, and the ends come out as +-1 by themselves
// (2^z = inf or 0).  The error stays below 2^-21 of the cap, whatever y is (in
// 2^-24 of it, at the worst y: ex2's 2^-22 and z's two roundings 2, the sum 1.7,
// rcp's last place 2, the last step 1.4): 2^-15 of a score's unit under a cap of
// 64, about a weight's own rounding to its 16-bit pair, and 2^-11 under the widest
// cap, 2^10, where it is what limits a 32-bit output.  (The series for small y
// would keep every bit under wide caps too; it cost the E4M3 decode 9 % and the
// prefill kernel registers.)
__device__ __forceinline__ float cap_score(float x, float z_of_x, float cap_log2) {
  return fmaf(rcp(1.f + ex2(x * z_of_x)), -2.f * cap_log2, cap_log2);
}

// Softmax weights meet V as pairs of 16-bit values, hi + lo.  Pairs of bf16 keep 16
// bits of any weight; those of fp16 end at 2^-24, and a weight relative to the row's
// largest score would be nothing below 2^-25: behind a first token that scores 17.4
// nats above 32767 others, all they bring.  So under fp16 the running reference stays
// kRefBelow under the largest score, in log2 units.  Scores may outgrow it by 2^8 before
// the next rescale: weights reach 2^15, and fp16 65504.
template <bool IsBF16>
constexpr float kRefBelow = IsBF16 ? 0.f : 7.f;
// The decode kernels leave it out under up to 16 pages, whose weights lose 2^-17 of the
// largest together, less than the pairs' own roundings: there the largest weighs exactly
// 1, and a sequence of one token gives its V row as it is.
__device__ __forceinline__ float ref_below(int pages) {
  return pages > 16 ? kRefBelow<false> : 0.f;
}

// Per-token E4M3: a row's V scale goes into its weight, and the pair of fp16 values
// needs their product in fp16's range whatever size V is.  So weights are relative to a
// reference that holds, beside the largest score, a power of two (the unit) that no V
// scale seen so far exceeds: it starts at the least one, and a larger scale moves it up
// as a larger score does.  l and o share the reference as ever.  (Without it V rows of
// 2^-10 came out 0.5 % off, and rows above 2^17 as infinities.)  Units span 2^124, so that
// a step from the least to the most still leaves of l, in fp32, what weighs more than
// 2^-25 of the rest.  64 x 8192 tokens take 201.0 us as before; with o in units of its
// own and the scales divided by them 204.0.
constexpr float kLeastUnit = 0x1p-40f, kMostUnit = 0x1p84f;
__device__ __forceinline__ float unit_above(uint32_t top) {  // top: a float >= 0, its bits
  return fminf(fmaxf(__uint_as_float(((top >> 23) + 1) << 23), kLeastUnit), kMostUnit);
}
__device__ __forceinline__ float log2_of_unit(float unit) {
  return (float)((int)(__float_as_uint(unit) >> 23) - 127);
}

// Two fp32 -> packed 16-bit pair (lo in the low half), round to nearest even.
template <bool IsBF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (IsBF16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
}

template <bool IsBF16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (IsBF16) {
    __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&u);
    return __bfloat1622float2(v);
  } else {
    __half2 v = *reinterpret_cast<__half2*>(&u);
    return __half22float2(v);
  }
}

// Two E4M3 bytes (low byte -> low half) to an exact fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_bytes) {
  uint32_t d;
  uint16_t s = static_cast<uint16_t>(two_bytes);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(s));
  return d;
}

// Two fp32 -> two E4M3 bytes, round to nearest even, saturating to +-448.
// `lo` lands in the low byte.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// Eight 16-bit values (one uint4) -> eight E4M3 bytes: each divided by
// `scale` in IEEE fp32, then encoded round-to-nearest-even with saturation.
template <bool IN_BF16>
__device__ __forceinline__ uint2 quantize8(uint4 in, float scale) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  uint32_t outw[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = unpack2<IN_BF16>(w[2 * i]);
    const float2 b = unpack2<IN_BF16>(w[2 * i + 1]);
    const uint16_t lo = f32x2_to_e4m3x2(__fdiv_rn(a.x, scale), __fdiv_rn(a.y, scale));
    const uint16_t hi = f32x2_to_e4m3x2(__fdiv_rn(b.x, scale), __fdiv_rn(b.y, scale));
    outw[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  return make_uint2(outw[0], outw[1]);
}

}  // namespace pkv
