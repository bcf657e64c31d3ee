// pkv_api.cu -- the C ABI (include/pkv.h): argument validation, launch
// sizing, tensor-map encoding and kernel dispatch.  No allocation, no
// synchronisation, no state beyond a per-device SM-count cache.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <atomic>
#include <mutex>

#include "pkv.h"
#include "pkv_internal.h"
#include "pkv_prefix_line.h"

namespace {

using pkv::kPageSize;

constexpr int kMaxDevices = 64;
std::atomic<int> g_sm_count[kMaxDevices];

int sm_count_current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return -1;
  if (dev < kMaxDevices) {
    int cached = g_sm_count[dev].load(std::memory_order_relaxed);
    if (cached > 0) return cached;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return -1;
  if (dev < kMaxDevices) g_sm_count[dev].store(n, std::memory_order_relaxed);
  return n;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Shape checks shared by both calls.
pkv_status check_desc(const pkv_cache_desc* d) {
  if (d == nullptr || d->struct_size != sizeof(pkv_cache_desc)) return PKV_ERR_INVALID_ARG;
  if (d->num_blocks <= 0 || d->page_size <= 0 || d->num_kv_heads <= 0 ||
      d->num_q_heads <= 0 || d->head_dim <= 0)
    return PKV_ERR_INVALID_ARG;
  if (d->num_q_heads % d->num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  if (d->page_size != kPageSize) return PKV_ERR_UNSUPPORTED;
  const int g = d->num_q_heads / d->num_kv_heads;
  if (g != 1 && g != 2 && g != 4 && g != 8) return PKV_ERR_UNSUPPORTED;
  switch (d->cache_dtype) {
    case PKV_F16:
    case PKV_BF16:
      if (d->head_dim != 64 && d->head_dim != 128) return PKV_ERR_UNSUPPORTED;
      break;
    case PKV_FP8_E4M3:
    case PKV_FP8_E4M3_TOKEN:
      if (d->head_dim != 128) return PKV_ERR_UNSUPPORTED;
      if (d->k_scale == nullptr) return PKV_ERR_INVALID_ARG;
      if (d->cache_dtype == PKV_FP8_E4M3 && d->v_scale == nullptr) return PKV_ERR_INVALID_ARG;
      // per token: one pool, a page's scales copied as one 128-byte line
      if (d->cache_dtype == PKV_FP8_E4M3_TOKEN && !aligned(d->k_scale, 128))
        return PKV_ERR_INVALID_ARG;
      break;
    default:
      return PKV_ERR_UNSUPPORTED;
  }
  const int64_t rows = (int64_t)d->num_blocks * d->num_kv_heads * d->page_size;
  if (rows >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

pkv::CacheKind kind_of(pkv_dtype t) {
  switch (t) {
    case PKV_FP8_E4M3: return pkv::kCacheE4M3;
    case PKV_FP8_E4M3_TOKEN: return pkv::kCacheE4M3Tok;
    case PKV_BF16: return pkv::kCacheBF16;
    default: return pkv::kCacheF16;
  }
}
bool is_fp8(pkv_dtype t) { return t == PKV_FP8_E4M3 || t == PKV_FP8_E4M3_TOKEN; }

struct WsLayout {
  size_t ml_off, o_off, ticket_bytes, total;
  int ctas;
};

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace: from the front, the split partials (one slot per CTA of the
// largest grid plus one per segment, slot cta + seg, each with room for the
// (query token, head) columns of a group: 8, or group x query tokens when
// that is more); at the very end of the caller's buffer, one page ticket per
// segment.  Only the tickets must be zero when a call starts, and a completed
// call leaves them at zero.  The partials' size grows with the batch and the
// columns and the tickets sit at the end, so a workspace sized for batch B
// and q_len Q serves every call with the same descriptor, a batch of at most
// B and at most Q query tokens: a smaller call's tickets are the tail of a
// larger call's, and no call's partials reach the tickets of any such call.
int nc_of(const pkv_cache_desc* d, int32_t qlen) {
  const int g = d->num_q_heads / d->num_kv_heads;
  const int qc = qlen <= 1 ? 1 : (qlen <= 2 ? 2 : (qlen <= 4 ? 4 : 8));
  return g * qc;
}
WsLayout ws_layout(const pkv_cache_desc* d, int32_t batch, int32_t mbs, int32_t hint,
                   int num_sms, int nc) {
  const int64_t g = pkv::decode_part_cols(nc);
  const int64_t cap = (int64_t)mbs * kPageSize;
  const int64_t len = (hint > 0 && hint < cap) ? hint : cap;
  const int64_t np_max = (len + kPageSize - 1) / kPageSize;
  const int64_t segs = (int64_t)batch * d->num_kv_heads;
  const int64_t pages_bound = segs * np_max;
  // at least eight pages per CTA (two per warp of a four-warp CTA); at most
  // kDecodeCtasPerSm CTAs per SM
  int64_t ctas = (pages_bound + 2 * pkv::kDecodeWarps - 1) / (2 * pkv::kDecodeWarps);
  const int64_t max_ctas = (int64_t)num_sms * pkv::kDecodeCtasPerSm;
  if (ctas > max_ctas) ctas = max_ctas;
  if (ctas < 1) ctas = 1;
  const int64_t slots = max_ctas + segs;
  WsLayout w;
  w.ctas = (int)ctas;
  w.ml_off = 0;
  w.o_off = align256(w.ml_off + (size_t)slots * g * 2 * sizeof(float));
  w.ticket_bytes = (size_t)segs * sizeof(int32_t);
  w.total = align256(w.o_off + (size_t)slots * g * d->head_dim * sizeof(float) + w.ticket_bytes);
  return w;
}

// The tickets of a call: the last ticket_bytes of the caller's buffer.
size_t ticket_offset(size_t workspace_bytes, const WsLayout& w) {
  return (workspace_bytes & ~(size_t)3) - w.ticket_bytes;
}

}  // namespace

namespace pkv {
cudaError_t decode_workspace_clear(void* workspace, size_t workspace_bytes,
                                   const pkv_cache_desc* d, int32_t batch, int32_t mbs,
                                   int32_t hint, cudaStream_t stream) {
  int sms = 0, dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const WsLayout w = ws_layout(d, batch, mbs, hint, sms, nc_of(d, 1));
  char* ws = static_cast<char*>(workspace);
  return cudaMemsetAsync(ws + ticket_offset(workspace_bytes, w), 0, w.ticket_bytes, stream);
}
}  // namespace pkv

namespace {

pkv_status encode_cache_map(CUtensorMap* map, const void* cache, const pkv_cache_desc* d) {
  auto fn = encode_fn();
  if (fn == nullptr) return PKV_ERR_CUDA;
  const bool fp8 = is_fp8(d->cache_dtype);
  const cuuint64_t elem = fp8 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)d->head_dim,
                              (cuuint64_t)d->num_blocks * d->num_kv_heads * d->page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)d->head_dim * elem};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / elem), (cuuint32_t)d->page_size};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                  const_cast<void*>(cache), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PKV_OK : PKV_ERR_CUDA;
}

// Query rows [rows][Hq][d] in boxes of 128 / g rows x the g heads of a KV head.
pkv_status encode_q_map(CUtensorMap* map, const void* q, const pkv_cache_desc* desc,
                        int32_t rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return PKV_ERR_CUDA;
  const cuuint64_t hd = (cuuint64_t)desc->head_dim;
  const cuuint64_t dims[3] = {hd, (cuuint64_t)desc->num_q_heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {hd * 2, (cuuint64_t)desc->num_q_heads * hd * 2};
  const int G = desc->num_q_heads / desc->num_kv_heads;
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(128 / G)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(q), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? PKV_OK
             : PKV_ERR_CUDA;
}

// A cap is 0 (none) or between 2^-10 and 2^10: the tanh's error is up to 2^-21 of
// the cap, so under a wider one a score could be more than 2^-11 off.
pkv_status bias_checks(float softcap, const float* slopes) {
  if (softcap != 0.f && !(softcap >= 0x1p-10f && softcap <= 0x1p10f)) return PKV_ERR_INVALID_ARG;
  if (!aligned(slopes, 4)) return PKV_ERR_INVALID_ARG;
  return PKV_OK;
}

// Shared prefix: the front of the workspace.  Sizes grow with the batch alone
// (the prefix's partials: one slot per CTA and segment; the own parts': one per
// chunk), so a workspace for a batch serves smaller ones.
constexpr int64_t kOwnItems = 4096;  // chunks of own parts over the batch, about
constexpr int32_t kOwnPages = 8;     // pages of a chunk, at least
struct SharedLayout {
  size_t pre_ml, pre_o, own_ml, own_o, total;
  int32_t pairs;
};
SharedLayout shared_layout(const pkv_cache_desc* d, int32_t batch, int sms) {
  const int64_t g = d->num_q_heads / d->num_kv_heads;
  const int64_t segs = (int64_t)batch * d->num_kv_heads;
  SharedLayout s;
  s.pairs = pkv::prefix_pairs((int64_t)batch * g);
  const int64_t pre_rows = ((int64_t)sms + (int64_t)s.pairs * d->num_kv_heads) * 256;
  const int64_t own_rows = (segs > kOwnItems ? segs : kOwnItems) * g;
  s.pre_ml = 256;
  s.pre_o = align256(s.pre_ml + pre_rows * 2 * sizeof(float));
  s.own_ml = align256(s.pre_o + pre_rows * d->head_dim * sizeof(float));
  s.own_o = align256(s.own_ml + own_rows * 2 * sizeof(float));
  s.total = align256(s.own_o + own_rows * d->head_dim * sizeof(float));
  return s;
}

// Whether the prefix is worth a pass of its own.  Otherwise one kernel reads it
// for every sequence, from L2 after the first, which takes 12 to 16 us and 0.1 us
// per MB read again; the three kernels take 12 to 16 us with a prefix of up to
// 1024 tokens, the prefix's one pass on top of that when it is longer, and more
// of the host's time (14 against 8 us).  Measured, one kernel against three, 32/8
// heads of 128: 4 x 4096 tokens 16.9 / 16.9 us, 8 x 1024 13.8 / 13.3, 32 x 256
// 17.5 / 15.6, 8 x 4096 22 / 17, 64 x 4096 106 / 28; two sequences never gain
// (2 x 16384: 24 / 29).
bool shared_pays(const pkv_cache_desc* d, int32_t batch, int32_t npb) {
  const int64_t again = (int64_t)(batch - 1) * npb * kPageSize * d->num_kv_heads * d->head_dim * 4;
  return batch >= 4 && again >= (int64_t)32 << 20;
}

pkv_status append_checks(const pkv_cache_desc* desc, const void* k_cache, const void* v_cache,
                         const int64_t* slot_mapping, const void* k, const void* v,
                         int32_t num_tokens, pkv_dtype kv_dtype) {
  if (!k_cache || !v_cache || !slot_mapping || !k || !v) return PKV_ERR_INVALID_ARG;
  if (kv_dtype != PKV_F16 && kv_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (!is_fp8(desc->cache_dtype) && kv_dtype != desc->cache_dtype)
    return PKV_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(slot_mapping, 8))
    return PKV_ERR_INVALID_ARG;
  (void)num_tokens;
  return PKV_OK;
}

pkv_status decode_checks(const pkv_cache_desc* desc, const void* q, const void* k_cache,
                         const void* v_cache, const int32_t* block_tables,
                         const int32_t* context_lens, int32_t batch, int32_t max_blocks_per_seq,
                         int32_t max_context_len_hint, float scale, const void* out,
                         pkv_dtype q_dtype, pkv_dtype out_dtype, const void* workspace,
                         size_t workspace_bytes, int32_t qlen = 1) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (batch < 0 || max_blocks_per_seq <= 0 || max_context_len_hint < 0)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0) return PKV_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
    return PKV_ERR_INVALID_ARG;
  if ((int64_t)batch * max_blocks_per_seq >= ((int64_t)1 << 31)) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * kPageSize >= ((int64_t)1 << 31)) return PKV_ERR_UNSUPPORTED;
  if (q_dtype != PKV_F16 && q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (!is_fp8(desc->cache_dtype) && q_dtype != desc->cache_dtype)
    return PKV_ERR_INVALID_ARG;
  if (out_dtype != PKV_F16 && out_dtype != PKV_BF16 && out_dtype != PKV_F32)
    return PKV_ERR_UNSUPPORTED;
  if (!(scale == scale)) return PKV_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4))
    return PKV_ERR_INVALID_ARG;
  if (qlen < 1 || qlen > 8) return PKV_ERR_UNSUPPORTED;
  const pkv::CacheKind cache = kind_of(desc->cache_dtype);
  const int nc = nc_of(desc, qlen);
  const size_t smem = qlen == 1 ? pkv::decode_smem_bytes(desc->head_dim, cache, batch)
                                 : pkv::mq_smem_bytes(desc->head_dim, cache, batch, nc);
  if (smem > 227 * 1024) return PKV_ERR_UNSUPPORTED;
  const int sms = sm_count_current_device();
  if (sms <= 0) return PKV_ERR_CUDA;
  const WsLayout w = ws_layout(desc, batch, max_blocks_per_seq, max_context_len_hint, sms, nc);
  if (workspace == nullptr || workspace_bytes < w.total || !aligned(workspace, 256))
    return PKV_ERR_WORKSPACE;
  return PKV_OK;
}

}  // namespace

namespace pkv {
pkv_status decode_validate(const pkv_cache_desc* desc, const void* q, const void* k_cache,
                           const void* v_cache, const int32_t* block_tables,
                           const int32_t* context_lens, int32_t batch, int32_t max_blocks_per_seq,
                           int32_t max_context_len_hint, float scale, const void* out,
                           pkv_dtype q_dtype, pkv_dtype out_dtype, const void* workspace,
                           size_t workspace_bytes) {
  return decode_checks(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                       max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype, out_dtype,
                       workspace, workspace_bytes);
}
}  // namespace pkv

namespace {

// What the biased and shared-prefix forms of the single-token kernel add.
struct DecodeForm {
  int mode = pkv::kModePlain;
  float softcap = 0.f;
  const float* slopes = nullptr;
  const int32_t* prefix_blocks = nullptr;
  int32_t npb = 0;
};

pkv_status decode_impl(const pkv_cache_desc* desc, const void* q, const void* k_cache,
                       const void* v_cache, const int32_t* block_tables,
                       const int32_t* context_lens, int32_t batch, int32_t max_blocks_per_seq,
                       int32_t max_context_len_hint, float scale, void* out, pkv_dtype q_dtype,
                       pkv_dtype out_dtype, void* workspace, size_t workspace_bytes,
                       pkv_stream_t stream, int early_prologue, int32_t qlen = 1,
                       int32_t window = 0, int32_t sinks = 0, const void* k_new = nullptr,
                       const void* v_new = nullptr, pkv_dtype kv_dtype = PKV_BF16,
                       int trigger_next = 0, const DecodeForm& form = DecodeForm()) {
  pkv_status st = decode_checks(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                                max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype,
                                out_dtype, workspace, workspace_bytes, qlen);
  if (st != PKV_OK || batch == 0) return st;
  const int sms = sm_count_current_device();
  const WsLayout w =
      ws_layout(desc, batch, max_blocks_per_seq, max_context_len_hint, sms, nc_of(desc, qlen));
  pkv::DecodeLaunch l;
  st = encode_cache_map(&l.tmap_k, k_cache, desc);
  if (st != PKV_OK) return st;
  st = encode_cache_map(&l.tmap_v, v_cache, desc);
  if (st != PKV_OK) return st;
  char* ws = static_cast<char*>(workspace);
  l.p.q = q;
  l.p.block_tables = block_tables;
  l.p.context_lens = context_lens;
  l.p.out = out;
  l.p.tickets = reinterpret_cast<int32_t*>(ws + ticket_offset(workspace_bytes, w));
  l.p.part_ml = reinterpret_cast<float*>(ws + w.ml_off);
  l.p.part_o = reinterpret_cast<float*>(ws + w.o_off);
  l.p.k_scale = desc->k_scale;
  l.p.v_scale = desc->v_scale;
  l.p.err_word = desc->err_word;
  l.p.B = batch;
  l.p.Hq = desc->num_q_heads;
  l.p.Hkv = desc->num_kv_heads;
  l.p.d = desc->head_dim;
  l.p.NB = desc->num_blocks;
  l.p.MBS = max_blocks_per_seq;
  l.p.out_dtype = out_dtype;
  l.p.early_prologue = early_prologue;
  l.p.trigger_next = trigger_next;
  l.p.qlen = qlen;
  l.p.window = window;
  l.p.k_new = k_new;
  l.p.v_new = v_new;
  l.p.k_cache = const_cast<void*>(k_cache);
  l.p.v_cache = const_cast<void*>(v_cache);
  l.p.kv_bf16 = kv_dtype == PKV_BF16 ? 1 : 0;
  l.p.sinks = window > 0 ? sinks : 0;
  l.p.scale_log2 = scale * 1.4426950408889634f;
  l.p.cap_log2 = form.softcap * 1.4426950408889634f;
  l.p.cap_z = form.softcap > 0.f ? 2.f / form.softcap : 0.f;
  l.p.slopes = form.slopes;
  l.p.prefix_blocks = form.prefix_blocks;
  l.p.npb = form.npb;
  l.group = desc->num_q_heads / desc->num_kv_heads;
  // query-token capacity of the kernel: 1, or the smallest of 2, 4, 8 that
  // holds qlen
  l.qcap = nc_of(desc, qlen) / l.group;
  l.cache = kind_of(desc->cache_dtype);
  l.q_bf16 = (q_dtype == PKV_BF16);
  l.ctas = w.ctas;
  l.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (form.mode == pkv::kModeShared) {
    e = l.cache == pkv::kCacheF16 ? pkv::launch_decode_shared_f16(l)
                                  : pkv::launch_decode_shared_bf16(l);
  } else if (form.mode == pkv::kModeCap) {
    switch (l.cache) {
      case pkv::kCacheF16: e = pkv::launch_decode_cap_f16(l); break;
      case pkv::kCacheBF16: e = pkv::launch_decode_cap_bf16(l); break;
      case pkv::kCacheE4M3: e = pkv::launch_decode_cap_e4m3(l); break;
      default: e = pkv::launch_decode_cap_e4m3_tok(l); break;
    }
  } else if (form.mode == pkv::kModeDist) {
    switch (l.cache) {
      case pkv::kCacheF16: e = pkv::launch_decode_dist_f16(l); break;
      case pkv::kCacheBF16: e = pkv::launch_decode_dist_bf16(l); break;
      case pkv::kCacheE4M3: e = pkv::launch_decode_dist_e4m3(l); break;
      default: e = pkv::launch_decode_dist_e4m3_tok(l); break;
    }
  } else if (l.qcap == 1) {
    switch (l.cache) {
      case pkv::kCacheF16: e = pkv::launch_decode_f16(l); break;
      case pkv::kCacheBF16: e = pkv::launch_decode_bf16(l); break;
      case pkv::kCacheE4M3: e = pkv::launch_decode_e4m3(l); break;
      default: e = pkv::launch_decode_e4m3_tok(l); break;
    }
  } else {
    switch (l.cache) {
      case pkv::kCacheF16: e = pkv::launch_decode_multi_f16(l); break;
      case pkv::kCacheBF16: e = pkv::launch_decode_multi_bf16(l); break;
      case pkv::kCacheE4M3: e = pkv::launch_decode_multi_e4m3(l); break;
      default: e = pkv::launch_decode_multi_e4m3_tok(l); break;
    }
  }
  if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

extern "C" {

pkv_status pkv_kv_append(const pkv_cache_desc* desc, void* k_cache, void* v_cache,
                         const int64_t* slot_mapping, const void* k, const void* v,
                         int32_t num_tokens, pkv_dtype kv_dtype, pkv_stream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  st = append_checks(desc, k_cache, v_cache, slot_mapping, k, v, num_tokens, kv_dtype);
  if (st != PKV_OK) return st;
  pkv::AppendParams a;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.slot_mapping = slot_mapping;
  a.block_tables = nullptr;
  a.context_lens = nullptr;
  a.MBS = 0;
  a.scale_out = nullptr;
  if (desc->cache_dtype == PKV_FP8_E4M3_TOKEN)  // the scale pool takes the rows' scales
    a.scale_out = const_cast<float*>(desc->k_scale);
  a.k = k;
  a.v = v;
  a.k_scale = desc->k_scale;
  a.v_scale = desc->v_scale;
  a.err_word = desc->err_word;
  a.T = num_tokens;
  a.Hkv = desc->num_kv_heads;
  a.d = desc->head_dim;
  a.NB = desc->num_blocks;
  cudaError_t e = pkv::launch_append(a, kind_of(desc->cache_dtype), kv_dtype == PKV_BF16,
                                     reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_kv_append_rope(const pkv_cache_desc* desc, void* k_cache, void* v_cache,
                              const int64_t* slot_mapping, const int64_t* positions,
                              const float* cos_sin, int32_t max_position, int32_t rot_dim,
                              const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, void* q_out, int32_t num_tokens,
                              pkv_dtype dtype, int32_t flags, pkv_stream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || (flags & ~PKV_ROPE_INTERLEAVED) != 0) return PKV_ERR_INVALID_ARG;
  if (rot_dim <= 0 || rot_dim > desc->head_dim || max_position <= 0) return PKV_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  st = append_checks(desc, k_cache, v_cache, slot_mapping, k, v, num_tokens, dtype);
  if (st != PKV_OK) return st;
  if (!positions || !cos_sin || !q || !q_out) return PKV_ERR_INVALID_ARG;
  if (!aligned(positions, 8) || !aligned(cos_sin, 16) || !aligned(q, 16) || !aligned(q_out, 16))
    return PKV_ERR_INVALID_ARG;
  const int64_t qrow = (int64_t)desc->num_q_heads * desc->head_dim;
  const int64_t kvrow = (int64_t)desc->num_kv_heads * desc->head_dim;
  if (q_stride < qrow || k_stride < kvrow || v_stride < kvrow) return PKV_ERR_INVALID_ARG;
  if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0) return PKV_ERR_INVALID_ARG;
  pkv::RopeParams p;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.slot_mapping = slot_mapping;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.k_scale = desc->k_scale;
  p.v_scale = desc->v_scale;
  p.scale_out = nullptr;
  if (desc->cache_dtype == PKV_FP8_E4M3_TOKEN) p.scale_out = const_cast<float*>(desc->k_scale);
  p.err_word = desc->err_word;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.T = num_tokens;
  p.Hq = desc->num_q_heads;
  p.Hkv = desc->num_kv_heads;
  p.d = desc->head_dim;
  p.NB = desc->num_blocks;
  p.rot = rot_dim;
  p.max_position = max_position;
  p.interleaved = (flags & PKV_ROPE_INTERLEAVED) ? 1 : 0;
  const cudaError_t e =
      pkv::launch_rope_append(p, kind_of(desc->cache_dtype), dtype == PKV_BF16,
                              reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_copy_blocks(const pkv_cache_desc* desc, void* k_cache, void* v_cache,
                           const int32_t* src_blocks, const int32_t* dst_blocks, int32_t n,
                           pkv_stream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (n < 0) return PKV_ERR_INVALID_ARG;
  if (n == 0) return PKV_OK;
  if (!k_cache || !v_cache || !src_blocks || !dst_blocks) return PKV_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(src_blocks, 4) ||
      !aligned(dst_blocks, 4))
    return PKV_ERR_INVALID_ARG;
  pkv::CopyParams c;
  c.k_cache = k_cache;
  c.v_cache = v_cache;
  c.src = src_blocks;
  c.dst = dst_blocks;
  c.err_word = desc->err_word;
  c.block_bytes = (int64_t)desc->num_kv_heads * desc->page_size * desc->head_dim *
                  (is_fp8(desc->cache_dtype) ? 1 : 2);
  c.scales = nullptr;  // per-token scales travel with their block
  if (desc->cache_dtype == PKV_FP8_E4M3_TOKEN) c.scales = const_cast<float*>(desc->k_scale);
  c.scales_per_block = desc->num_kv_heads * 2 * desc->page_size;
  c.NB = desc->num_blocks;
  const cudaError_t e = pkv::launch_copy_blocks(c, n, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

size_t pkv_decode_workspace_bytes(const pkv_cache_desc* desc, int32_t batch,
                                  int32_t max_blocks_per_seq, int32_t max_context_len_hint) {
  return pkv_decode_workspace_bytes_multi(desc, batch, 1, max_blocks_per_seq,
                                          max_context_len_hint);
}

size_t pkv_decode_workspace_bytes_multi(const pkv_cache_desc* desc, int32_t batch,
                                        int32_t q_len, int32_t max_blocks_per_seq,
                                        int32_t max_context_len_hint) {
  if (check_desc(desc) != PKV_OK || batch < 0 || max_blocks_per_seq <= 0) return 0;
  if (q_len < 1 || q_len > 8) return 0;
  if (batch == 0) return 0;
  const int sms = sm_count_current_device();
  if (sms <= 0) return 0;
  return ws_layout(desc, batch, max_blocks_per_seq, max_context_len_hint, sms,
                   nc_of(desc, q_len)).total;
}

pkv_status pkv_paged_decode_attention(const pkv_cache_desc* desc, const void* q,
                                      const void* k_cache, const void* v_cache,
                                      const int32_t* block_tables, const int32_t* context_lens,
                                      int32_t batch, int32_t max_blocks_per_seq,
                                      int32_t max_context_len_hint, float scale, void* out,
                                      pkv_dtype q_dtype, pkv_dtype out_dtype, void* workspace,
                                      size_t workspace_bytes, pkv_stream_t stream) {
  return decode_impl(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                     max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype, out_dtype,
                     workspace, workspace_bytes, stream, /*early_prologue=*/0);
}

pkv_status pkv_paged_decode_attention_multi(
    const pkv_cache_desc* desc, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, int32_t batch, int32_t q_len,
    int32_t max_blocks_per_seq, int32_t max_context_len_hint, float scale, void* out,
    pkv_dtype q_dtype, pkv_dtype out_dtype, void* workspace, size_t workspace_bytes,
    pkv_stream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (q_len < 1) return PKV_ERR_INVALID_ARG;
  if (q_len > 8) return PKV_ERR_UNSUPPORTED;
  return decode_impl(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                     max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype, out_dtype,
                     workspace, workspace_bytes, stream, /*early_prologue=*/0, q_len);
}

pkv_status pkv_paged_decode_attention_window(
    const pkv_cache_desc* desc, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, int32_t batch, int32_t q_len,
    int32_t window, int32_t sinks, int32_t max_blocks_per_seq, int32_t max_context_len_hint,
    float scale, void* out, pkv_dtype q_dtype, pkv_dtype out_dtype, void* workspace,
    size_t workspace_bytes, pkv_stream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (q_len < 1 || window < 0 || sinks < 0) return PKV_ERR_INVALID_ARG;
  if (q_len > 8) return PKV_ERR_UNSUPPORTED;
  return decode_impl(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                     max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype, out_dtype,
                     workspace, workspace_bytes, stream, /*early_prologue=*/0, q_len, window,
                     sinks);
}

pkv_status pkv_decode_step(const pkv_cache_desc* desc, const void* q, void* k_cache,
                           void* v_cache, const int64_t* slot_mapping, const void* k,
                           const void* v, pkv_dtype kv_dtype, const int32_t* block_tables,
                           const int32_t* context_lens, int32_t batch,
                           int32_t max_blocks_per_seq, int32_t max_context_len_hint,
                           float scale, void* out, pkv_dtype q_dtype, pkv_dtype out_dtype,
                           void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  // Validate everything before the first launch, so an error launches nothing.
  pkv_status st = decode_checks(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                                max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype,
                                out_dtype, workspace, workspace_bytes);
  if (st != PKV_OK) return st;
  if (batch > 0) {
    st = append_checks(desc, k_cache, v_cache, slot_mapping, k, v, batch, kv_dtype);
    if (st != PKV_OK) return st;
  }
  st = pkv_kv_append(desc, k_cache, v_cache, slot_mapping, k, v, batch, kv_dtype, stream);
  if (st != PKV_OK) return st;
  return decode_impl(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                     max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype, out_dtype,
                     workspace, workspace_bytes, stream, /*early_prologue=*/1);
}

pkv_status pkv_paged_decode_attention_biased(
    const pkv_cache_desc* desc, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, int32_t batch, int32_t window,
    int32_t sinks, float softcap, const float* alibi_slopes, int32_t max_blocks_per_seq,
    int32_t max_context_len_hint, float scale, void* out, pkv_dtype q_dtype, pkv_dtype out_dtype,
    void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (window < 0 || sinks < 0) return PKV_ERR_INVALID_ARG;
  st = bias_checks(softcap, alibi_slopes);
  if (st != PKV_OK) return st;
  DecodeForm form;
  if (softcap > 0.f) form.mode = pkv::kModeCap;
  else if (alibi_slopes != nullptr) form.mode = pkv::kModeDist;
  form.softcap = softcap;
  form.slopes = alibi_slopes;
  return decode_impl(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                     max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype, out_dtype,
                     workspace, workspace_bytes, stream, /*early_prologue=*/0, 1, window, sinks,
                     nullptr, nullptr, PKV_BF16, 0, form);
}

size_t pkv_shared_prefix_workspace_bytes(const pkv_cache_desc* desc, int32_t batch,
                                         int32_t num_prefix_blocks, int32_t max_blocks_per_seq,
                                         int32_t max_context_len_hint) {
  if (check_desc(desc) != PKV_OK || is_fp8(desc->cache_dtype)) return 0;
  if (num_prefix_blocks < 0 || num_prefix_blocks > max_blocks_per_seq) return 0;
  const size_t own =
      pkv_decode_workspace_bytes(desc, batch, max_blocks_per_seq, max_context_len_hint);
  const int sms = sm_count_current_device();
  return own == 0 || sms <= 0 ? 0 : shared_layout(desc, batch, sms).total + own;
}

pkv_status pkv_paged_decode_attention_shared_prefix(
    const pkv_cache_desc* desc, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* prefix_blocks, int32_t num_prefix_blocks, const int32_t* block_tables,
    const int32_t* context_lens, int32_t batch, int32_t max_blocks_per_seq,
    int32_t max_context_len_hint, float scale, void* out, pkv_dtype q_dtype, pkv_dtype out_dtype,
    void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (is_fp8(desc->cache_dtype)) return PKV_ERR_UNSUPPORTED;
  if (num_prefix_blocks < 0 || num_prefix_blocks > max_blocks_per_seq) return PKV_ERR_INVALID_ARG;
  if (!(scale > 0.f)) return PKV_ERR_INVALID_ARG;  // row maxima are taken unscaled
  if (batch > 0 && num_prefix_blocks > 0 && (!prefix_blocks || !aligned(prefix_blocks, 4)))
    return PKV_ERR_INVALID_ARG;
  const int sms = sm_count_current_device();
  const SharedLayout s = shared_layout(desc, batch > 0 ? batch : 1, sms > 0 ? sms : 1);
  char* ws = static_cast<char*>(workspace);
  char* own = workspace_bytes > s.total && ws != nullptr ? ws + s.total : nullptr;
  const size_t own_bytes = own != nullptr ? workspace_bytes - s.total : 0;
  st = decode_checks(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                     max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype, out_dtype,
                     own, own_bytes);
  if (st != PKV_OK || batch == 0) return st;
  DecodeForm form;
  form.mode = pkv::kModeShared;
  form.prefix_blocks = prefix_blocks;
  form.npb = num_prefix_blocks;
  if (!shared_pays(desc, batch, num_prefix_blocks))
    return decode_impl(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                       max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype, out_dtype,
                       own, own_bytes, stream, /*early_prologue=*/0, 1, 0, 0, nullptr, nullptr,
                       PKV_BF16, 0, form);
  // the prefix for all rows at once, each sequence's own part, the merge
  pkv::PrefixLaunch l;
  st = encode_cache_map(&l.tmap_k, k_cache, desc);
  if (st != PKV_OK) return st;
  st = encode_cache_map(&l.tmap_v, v_cache, desc);
  if (st != PKV_OK) return st;
  st = encode_q_map(&l.tmap_q, q, desc, batch);
  if (st != PKV_OK) return st;
  l.p.q = q;
  l.p.context_lens = context_lens;
  l.p.prefix_blocks = prefix_blocks;
  l.p.block_tables = block_tables;
  l.p.out = out;
  l.p.seen = reinterpret_cast<int32_t*>(ws);
  l.p.pre_ml = reinterpret_cast<float2*>(ws + s.pre_ml);
  l.p.pre_o = reinterpret_cast<float*>(ws + s.pre_o);
  l.p.own_ml = reinterpret_cast<float2*>(ws + s.own_ml);
  l.p.own_o = reinterpret_cast<float*>(ws + s.own_o);
  l.p.err_word = desc->err_word;
  l.p.B = batch;
  l.p.Hq = desc->num_q_heads;
  l.p.Hkv = desc->num_kv_heads;
  l.p.NB = desc->num_blocks;
  l.p.MBS = max_blocks_per_seq;
  l.p.npb = num_prefix_blocks;
  l.p.pairs = s.pairs;
  const int64_t blocks = pkv::prefix_blocks_of((int64_t)num_prefix_blocks * kPageSize);
  const int64_t rows = (int64_t)batch * (desc->num_q_heads / desc->num_kv_heads);
  const int last_w = pkv::prefix_last_weight(rows, s.pairs);
  l.p.ctas = (int32_t)pkv::prefix_ctas(
      pkv::prefix_cost(desc->num_kv_heads, blocks, s.pairs, last_w), sms);
  l.sms = sms;
  // own parts are cut into chunks of kOwnPages pages or more, about kOwnItems in
  // all (from the longest own part the arguments allow: empty chunks are cheap)
  const int64_t cap = (int64_t)max_blocks_per_seq * kPageSize;
  const int64_t longest =
      max_context_len_hint > 0 && max_context_len_hint < cap ? max_context_len_hint : cap;
  int64_t most_own = (longest + kPageSize - 1) / kPageSize - num_prefix_blocks;
  if (most_own < 1) most_own = 1;
  const int64_t segs = (int64_t)batch * desc->num_kv_heads;
  int64_t chunks = kOwnItems / segs;
  if (chunks > (most_own + kOwnPages - 1) / kOwnPages)
    chunks = (most_own + kOwnPages - 1) / kOwnPages;
  if (chunks < 1) chunks = 1;
  l.p.chunks = (int32_t)chunks;
  l.p.chunk_pages = (int32_t)((most_own + chunks - 1) / chunks);
  l.p.out_dtype = out_dtype;
  l.p.scale_log2 = scale * 1.4426950408889634f;
  l.bf16 = desc->cache_dtype == PKV_BF16;
  l.d = desc->head_dim;
  l.stream = reinterpret_cast<cudaStream_t>(stream);
  if (segs * chunks >= ((int64_t)1 << 31)) return PKV_ERR_UNSUPPORTED;
  return pkv::launch_prefix(l) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"

namespace {
pkv_status prefill_impl(const pkv_cache_desc* desc, const void* q, const void* k_cache,
                        const void* v_cache, const int32_t* block_tables,
                        const int32_t* context_lens, const int32_t* q_start, int32_t batch,
                        int32_t total_q, int32_t max_q_len, int32_t max_blocks_per_seq,
                        float scale, float softcap, const float* slopes, void* out,
                        pkv_dtype q_dtype, pkv_dtype out_dtype, pkv_stream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (batch < 0 || total_q < 0 || max_q_len < 0 || max_blocks_per_seq <= 0)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0 || total_q == 0 || max_q_len == 0) return PKV_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !q_start || !out)
    return PKV_ERR_INVALID_ARG;
  if (desc->cache_dtype != PKV_F16 && desc->cache_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (desc->head_dim != 64 && desc->head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (q_dtype != desc->cache_dtype) return PKV_ERR_INVALID_ARG;
  if (out_dtype != PKV_F16 && out_dtype != PKV_BF16 && out_dtype != PKV_F32)
    return PKV_ERR_UNSUPPORTED;
  if (!(scale > 0.f)) return PKV_ERR_INVALID_ARG;  // the kernel takes row maxima unscaled
  if ((int64_t)batch * max_blocks_per_seq >= ((int64_t)1 << 31)) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * kPageSize >= ((int64_t)1 << 31)) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)total_q * desc->num_q_heads >= ((int64_t)1 << 31)) return PKV_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(q_start, 4))
    return PKV_ERR_INVALID_ARG;
  pkv::PrefillLaunch l;
  st = encode_cache_map(&l.tmap_k, k_cache, desc);
  if (st != PKV_OK) return st;
  st = encode_cache_map(&l.tmap_v, v_cache, desc);
  if (st != PKV_OK) return st;
  st = encode_q_map(&l.tmap_q, q, desc, total_q);
  if (st != PKV_OK) return st;
  const int G = desc->num_q_heads / desc->num_kv_heads;
  l.p.q_start = q_start;
  l.p.context_lens = context_lens;
  l.p.block_tables = block_tables;
  l.p.out = out;
  l.p.err_word = desc->err_word;
  l.p.B = batch;
  l.p.Hq = desc->num_q_heads;
  l.p.Hkv = desc->num_kv_heads;
  l.p.NB = desc->num_blocks;
  l.p.MBS = max_blocks_per_seq;
  l.p.total_q = total_q;
  l.p.tiles_per_seq = (max_q_len + 256 / G - 1) / (256 / G);  // a CTA: 256 / G tokens
  l.p.out_dtype = out_dtype;
  l.p.scale_log2 = scale * 1.4426950408889634f;
  l.p.cap_log2 = softcap * 1.4426950408889634f;
  l.p.cap_z = softcap > 0.f ? l.p.scale_log2 * (2.f / softcap) : 0.f;
  l.p.slopes = slopes;
  if (!(l.p.cap_z < INFINITY)) return PKV_ERR_INVALID_ARG;
  l.bf16 = desc->cache_dtype == PKV_BF16;
  l.d = desc->head_dim;
  l.stream = reinterpret_cast<cudaStream_t>(stream);
  if ((int64_t)batch * l.p.tiles_per_seq >= ((int64_t)1 << 31)) return PKV_ERR_UNSUPPORTED;
  const cudaError_t e = softcap > 0.f       ? pkv::launch_prefill_cap(l)
                        : slopes != nullptr ? pkv::launch_prefill_dist(l)
                                            : pkv::launch_prefill(l);
  if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
}  // namespace

extern "C" {

pkv_status pkv_paged_prefill_attention(const pkv_cache_desc* desc, const void* q,
                                       const void* k_cache, const void* v_cache,
                                       const int32_t* block_tables,
                                       const int32_t* context_lens, const int32_t* q_start,
                                       int32_t batch, int32_t total_q, int32_t max_q_len,
                                       int32_t max_blocks_per_seq, float scale, void* out,
                                       pkv_dtype q_dtype, pkv_dtype out_dtype,
                                       pkv_stream_t stream) {
  return prefill_impl(desc, q, k_cache, v_cache, block_tables, context_lens, q_start, batch,
                      total_q, max_q_len, max_blocks_per_seq, scale, 0.f, nullptr, out, q_dtype,
                      out_dtype, stream);
}

pkv_status pkv_paged_prefill_attention_biased(
    const pkv_cache_desc* desc, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, const int32_t* q_start,
    int32_t batch, int32_t total_q, int32_t max_q_len, int32_t max_blocks_per_seq, float scale,
    float softcap, const float* alibi_slopes, void* out, pkv_dtype q_dtype, pkv_dtype out_dtype,
    pkv_stream_t stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  st = bias_checks(softcap, alibi_slopes);
  if (st != PKV_OK) return st;
  return prefill_impl(desc, q, k_cache, v_cache, block_tables, context_lens, q_start, batch,
                      total_q, max_q_len, max_blocks_per_seq, scale, softcap, alibi_slopes, out,
                      q_dtype, out_dtype, stream);
}

pkv_status pkv_decode_step_fused(const pkv_cache_desc* desc, const void* q, void* k_cache,
                                 void* v_cache, const void* k, const void* v,
                                 pkv_dtype kv_dtype, const int32_t* block_tables,
                                 const int32_t* context_lens, int32_t batch,
                                 int32_t max_blocks_per_seq, int32_t max_context_len_hint,
                                 float scale, void* out, pkv_dtype q_dtype, pkv_dtype out_dtype,
                                 void* workspace, size_t workspace_bytes, int32_t flags,
                                 pkv_stream_t stream) {
  pkv_status st = decode_checks(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                                max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype,
                                out_dtype, workspace, workspace_bytes);
  if (st != PKV_OK || batch == 0) return st;
  if (!k || !v) return PKV_ERR_INVALID_ARG;
  if (kv_dtype != PKV_F16 && kv_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (!is_fp8(desc->cache_dtype) && kv_dtype != desc->cache_dtype)
    return PKV_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16)) return PKV_ERR_INVALID_ARG;
  if ((flags & ~PKV_STEP_OVERLAP) != 0) return PKV_ERR_INVALID_ARG;
  const int overlap = (flags & PKV_STEP_OVERLAP) ? 1 : 0;
  if (is_fp8(desc->cache_dtype)) {
    // E4M3: the append kernel (each sequence's newest position, from its
    // table), then the attention overlapping its tail
    pkv::AppendParams a;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.slot_mapping = nullptr;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.MBS = max_blocks_per_seq;
    a.scale_out = nullptr;
    if (desc->cache_dtype == PKV_FP8_E4M3_TOKEN) a.scale_out = const_cast<float*>(desc->k_scale);
    a.k = k;
    a.v = v;
    a.k_scale = desc->k_scale;
    a.v_scale = desc->v_scale;
    a.err_word = desc->err_word;
    a.T = batch;
    a.Hkv = desc->num_kv_heads;
    a.d = desc->head_dim;
    a.NB = desc->num_blocks;
    if (pkv::launch_append(a, kind_of(desc->cache_dtype), kv_dtype == PKV_BF16,
                           reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
      return PKV_ERR_CUDA;
    return decode_impl(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                       max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype, out_dtype,
                       workspace, workspace_bytes, stream, /*early_prologue=*/1, 1, 0, 0,
                       nullptr, nullptr, kv_dtype, /*trigger_next=*/overlap);
  }
  return decode_impl(desc, q, k_cache, v_cache, block_tables, context_lens, batch,
                     max_blocks_per_seq, max_context_len_hint, scale, out, q_dtype, out_dtype,
                     workspace, workspace_bytes, stream, /*early_prologue=*/overlap, 1, 0, 0, k,
                     v, kv_dtype, /*trigger_next=*/overlap);
}

uint64_t pkv_kv_bytes_per_token(int32_t layers, int32_t kv_heads, int32_t head_dim,
                                int32_t elem_bytes) {
  if (layers < 0 || kv_heads < 0 || head_dim < 0 || elem_bytes < 0) return 0;
  return 2ull * (uint64_t)layers * (uint64_t)kv_heads * (uint64_t)head_dim *
         (uint64_t)elem_bytes;
}

const char* pkv_status_string(pkv_status s) {
  switch (s) {
    case PKV_OK: return "PKV_OK";
    case PKV_ERR_INVALID_ARG: return "PKV_ERR_INVALID_ARG: invalid argument";
    case PKV_ERR_UNSUPPORTED: return "PKV_ERR_UNSUPPORTED: shape or dtype not built";
    case PKV_ERR_WORKSPACE: return "PKV_ERR_WORKSPACE: workspace missing, misaligned or too small";
    case PKV_ERR_CUDA: return "PKV_ERR_CUDA: CUDA call failed";
    case PKV_ERR_BOUNDS: return "PKV_ERR_BOUNDS: slot, block id or context length out of range";
    case PKV_ERR_TIMEOUT: return "PKV_ERR_TIMEOUT: a bounded device wait gave up";
  }
  return "unknown pkv_status";
}

int32_t pkv_version(void) { return 100; }

}  // extern "C"
