// Append with the rotary position embedding applied on the way: q and k are
// rotated by their token's position, q goes to q_out, k and v to their cache
// slots.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

// A head row of d elements is d / 16 items of two 16-byte chunks; one thread
// takes one item.  An item holds eight whole rotation pairs, so nothing but
// the per-token E4M3 scale crosses threads:
//   split halves  chunks i and i + R / 16 of the first R elements
//   interleaved   chunks 2 i and 2 i + 1
//   past R        chunks 2 i and 2 i + 1, copied
// and pair j of item i turns by the angle 8 i + j of its position's table row
// (R / 2 cosines, then R / 2 sines):
//   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin       in fp32, rounded once.
// An E4M3 row is encoded from the fp32 values.
template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<BF16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                    pack2<BF16>(x[6], x[7]));
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t lo =
        f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
    const uint16_t hi =
        f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
    w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Bound by HBM for many tokens, by latency for few.  A thread takes the same
// item of NR rows of one token: their loads go out together, and the item's 16
// cosines and sines (from L2) are read once for all of them.  8192 tokens of
// 64/8 heads of 128 (340 MB): 67.2, 59.3, 61.5, 55.9, 61.7, 59.2 us with 1, 2, 3,
// 4, 5, 8 rows (55.9: 6.08 TB/s).  Where one row per thread fits the GPU at once
// it is the shorter chain: 1 token 2.1 us against 2.7, 128 tokens of 32/8 heads
// 2.5 against 3.1, 512 3.9 against 3.9, 1024 5.9 against 4.8.  E4M3 rows, whose
// divisions want more threads, change over later: with per-token scales 128
// tokens 3.1 against 4.3, 1024 7.6 against 8.8, 2048 12.6 against 12.9.
constexpr int kRowsPer = 4;
constexpr int64_t kOneRowThreads = 1 << 17, kOneRowThreadsFp8 = 1 << 20;

template <int CACHE, bool BF16, int NR>
__global__ void __launch_bounds__(256) rope_append_kernel(const RopeParams p) {
  // let a dependent kernel start its prologue while this one runs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr bool kFp8 = cache_is_fp8((CacheKind)CACHE);
  const int items = p.d >> 4;  // per head row: 4 or 8
  const int rows = p.Hq + 2 * p.Hkv;  // q heads, then k heads, then v heads
  const int groups = (rows + NR - 1) / NR;  // row g, g + groups, ... go to one thread
  const int64_t unit = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / items;
  const int t = (int)(unit / groups);
  if (t >= p.T) return;  // whole rows: the lanes of a row go together
  const int g = (int)(unit - (int64_t)t * groups);
  const int i = threadIdx.x % items;  // blockDim.x is a multiple of the items
  const int64_t pos = p.positions[t];
  const int64_t slot = p.slot_mapping[t];
  const bool in_rot = i < (p.rot >> 4);
  const bool halves = in_rot && !p.interleaved;

  uint4 u0[NR], u1[NR];
#pragma unroll
  for (int k = 0; k < NR; ++k) {
    const int r = g + k * groups;
    if (r >= rows) continue;
    const int which = r < p.Hq ? 0 : (r < p.Hq + p.Hkv ? 1 : 2);
    const int h = r - (which == 0 ? 0 : which == 1 ? p.Hq : p.Hq + p.Hkv);
    const int64_t stride = which == 0 ? p.q_stride : which == 1 ? p.k_stride : p.v_stride;
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(which == 0 ? p.q : which == 1 ? p.k : p.v) + t * stride +
        (int64_t)h * p.d);
    const bool apart = halves && which != 2;
    u0[k] = src[apart ? i : 2 * i];
    u1[k] = src[apart ? i + (p.rot >> 4) : 2 * i + 1];
  }
  if (pos < 0 || pos >= p.max_position) {
    if (g == 0 && i == 0) report_error(p.err_word, PKV_ERR_BOUNDS);
    return;
  }
  float c[8], s[8];
  if (in_rot) {
    const float4* cs = reinterpret_cast<const float4*>(p.cos_sin + pos * p.rot);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 cv = cs[2 * i + j], sv = cs[(p.rot >> 3) + 2 * i + j];
      c[4 * j] = cv.x; c[4 * j + 1] = cv.y; c[4 * j + 2] = cv.z; c[4 * j + 3] = cv.w;
      s[4 * j] = sv.x; s[4 * j + 1] = sv.y; s[4 * j + 2] = sv.z; s[4 * j + 3] = sv.w;
    }
  }
  const bool stored = slot >= 0 && slot < (int64_t)p.NB * kPageSize;
  if (slot >= (int64_t)p.NB * kPageSize && g == 0 && i == 0)
    report_error(p.err_word, PKV_ERR_BOUNDS);
  const int64_t blk = slot / kPageSize, off = slot - blk * kPageSize;

#pragma unroll
  for (int k = 0; k < NR; ++k) {
    const int r = g + k * groups;
    if (r >= rows) continue;
    const int which = r < p.Hq ? 0 : (r < p.Hq + p.Hkv ? 1 : 2);
    if (which != 0 && !stored) continue;
    const int h = r - (which == 0 ? 0 : which == 1 ? p.Hq : p.Hq + p.Hkv);
    const bool turned = in_rot && which != 2, apart = halves && which != 2;
    const int c0 = apart ? i : 2 * i, c1 = apart ? i + (p.rot >> 4) : 2 * i + 1;
    float a[8], b[8];
    if (turned || kFp8) {
      unpack8<BF16>(u0[k], a);
      unpack8<BF16>(u1[k], b);
    }
    if (turned) {
      if (!p.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x0 = a[j], x1 = b[j];
          a[j] = fmaf(x0, c[j], -(x1 * s[j]));
          b[j] = fmaf(x1, c[j], x0 * s[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x0 = a[2 * j], x1 = a[2 * j + 1];
          a[2 * j] = fmaf(x0, c[j], -(x1 * s[j]));
          a[2 * j + 1] = fmaf(x1, c[j], x0 * s[j]);
          x0 = b[2 * j];
          x1 = b[2 * j + 1];
          b[2 * j] = fmaf(x0, c[4 + j], -(x1 * s[4 + j]));
          b[2 * j + 1] = fmaf(x1, c[4 + j], x0 * s[4 + j]);
        }
      }
      if (which == 0 || !kFp8) {
        u0[k] = pack8<BF16>(a);
        u1[k] = pack8<BF16>(b);
      }
    }
    if (which == 0) {
      uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) +
                                            ((int64_t)t * p.Hq + h) * p.d);
      out[c0] = u0[k];
      out[c1] = u1[k];
      continue;
    }
    const int64_t dst = ((blk * p.Hkv + h) * kPageSize + off) * (p.d >> 3);
    void* cache = which == 1 ? p.k_cache : p.v_cache;
    if constexpr (!kFp8) {
      reinterpret_cast<uint4*>(cache)[dst + c0] = u0[k];
      reinterpret_cast<uint4*>(cache)[dst + c1] = u1[k];
    } else {
      float scale;
      if constexpr (CACHE == kCacheE4M3) {
        scale = (which == 1 ? p.k_scale : p.v_scale)[h];
      } else {
        // the row's own scale: its largest magnitude over 448 in IEEE fp32 (1
        // for an all-zero row); a row is eight neighbouring lanes (d = 128)
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(a[j]), fabsf(b[j])));
        const unsigned lanes = 0xffu << (threadIdx.x & 24);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o));
        scale = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
        // pool [NB][Hkv][2][P]: the page's K scales, then its V scales
        if (i == 0)
          p.scale_out[(blk * p.Hkv + h) * 2 * kPageSize + (which == 2 ? kPageSize : 0) + off] =
              scale;
      }
      reinterpret_cast<uint2*>(cache)[dst + c0] = encode8(a, scale);
      reinterpret_cast<uint2*>(cache)[dst + c1] = encode8(b, scale);
    }
  }
}

template <int NR>
cudaError_t launch_rope(const RopeParams& p, CacheKind cache, bool bf16, cudaStream_t stream) {
  const int64_t threads = (int64_t)p.T * ((p.Hq + 2 * p.Hkv + NR - 1) / NR) * (p.d / 16);
  const int block = 256;
  const int64_t grid = (threads + block - 1) / block;
  if (grid > 0x7fffffff) return cudaErrorNotSupported;
  auto kern = rope_append_kernel<kCacheBF16, true, NR>;
  if (cache == kCacheE4M3)
    kern = bf16 ? rope_append_kernel<kCacheE4M3, true, NR>
                : rope_append_kernel<kCacheE4M3, false, NR>;
  else if (cache == kCacheE4M3Tok)
    kern = bf16 ? rope_append_kernel<kCacheE4M3Tok, true, NR>
                : rope_append_kernel<kCacheE4M3Tok, false, NR>;
  else if (!bf16)
    kern = rope_append_kernel<kCacheF16, false, NR>;
  kern<<<(unsigned)grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rope_append(const RopeParams& p, CacheKind cache, bool bf16,
                               cudaStream_t stream) {
  const int64_t threads = (int64_t)p.T * (p.Hq + 2 * p.Hkv) * (p.d / 16);
  const bool one = threads <= (cache_is_fp8(cache) ? kOneRowThreadsFp8 : kOneRowThreads);
  return one ? launch_rope<1>(p, cache, bf16, stream)
             : launch_rope<kRowsPer>(p, cache, bf16, stream);
}

}  // namespace pkv
