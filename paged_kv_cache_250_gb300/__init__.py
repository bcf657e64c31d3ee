"""Python binding of libpkv.so: paged-KV single-token decode attention for GB300.

Argument marshalling only.  Every step of the decode path runs in the CUDA
kernels behind the C ABI declared in ``include/pkv.h``; torch supplies device
memory and streams.  The functions carry the C names:

    pkv_kv_append                 write new K/V rows into their cache slots
    pkv_kv_append_rope            the same with q and k rotated by their
                                  positions (rotary embedding) on the way
    pkv_decode_workspace_bytes    workspace size for a decode call
    pkv_decode_workspace_bytes_multi  the same for q_len query tokens per
                                  sequence (multi-query and windowed calls)
    pkv_paged_decode_attention    one (1,N) attention row per query head
    pkv_paged_decode_attention_multi  q_len new tokens per sequence, causal
    pkv_paged_decode_attention_window  the same under a sliding window with
                                  attention sinks
    pkv_paged_decode_attention_biased  decode with scores capped by a tanh, a
                                  distance bias, or both
    pkv_paged_decode_attention_scored  decode that adds up the attention weight
                                  each cached row receives
    pkv_scored_workspace_bytes    workspace size for that call
    pkv_kv_evict                  keep the rows with the largest weights, the
                                  first and the most recent ones
    pkv_paged_tree_attention      a tree of drafted tokens per sequence (tcgen05)
    pkv_tree_workspace_bytes      workspace size for that call
    pkv_kv_accept_path            keep the rows of a path through the tree
    pkv_paged_decode_attention_shared_prefix  decode for a batch whose
                                  sequences begin with the same blocks, read
                                  once for every 256 query rows of a KV head
    pkv_shared_prefix_workspace_bytes  workspace size for that call
    pkv_paged_prefill_attention   a chunk of new tokens per sequence, causal,
                                  on the tensor cores (tcgen05)
    pkv_paged_prefill_attention_biased  the same with capped or biased scores
    pkv_decode_step               both, validated together, the attention
                                  kernel overlapping the append's tail
    pkv_decode_step_fused         both in one kernel (new token at its
                                  sequence's newest position)
    pkv_copy_blocks               copy whole blocks (copy-on-write of a
                                  shared prefix's last block)
    pkv_paged_decode_attention_noalloc  decode without a caller workspace
    pkv_kv_bytes_per_token        cache bytes per token (host helper)
    pkv_status_string, pkv_version

If the library is missing it is built on first use with nvcc; if that is not
possible every call raises.  There is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

from . import build as _build

__all__ = [
    "PkvError", "CacheDesc", "make_desc", "load_library", "library_path",
    "pkv_kv_append", "pkv_decode_workspace_bytes", "pkv_paged_decode_attention",
    "pkv_decode_step", "pkv_kv_bytes_per_token", "pkv_status_string", "pkv_version",
    "pkv_paged_decode_attention_noalloc", "PKV_NOALLOC_SCRATCH_BYTES", "pkv_copy_blocks",
    "pkv_decode_workspace_bytes_multi",
    "pkv_paged_decode_attention_multi", "pkv_paged_decode_attention_window",
    "pkv_decode_step_fused", "pkv_paged_prefill_attention", "pkv_kv_append_rope",
    "pkv_paged_decode_attention_biased", "pkv_paged_prefill_attention_biased",
    "pkv_paged_decode_attention_shared_prefix", "pkv_shared_prefix_workspace_bytes",
    "pkv_paged_decode_attention_scored", "pkv_scored_workspace_bytes", "pkv_kv_evict",
    "pkv_paged_tree_attention", "pkv_tree_workspace_bytes", "pkv_kv_accept_path",
    "PKV_MAX_TREE",
    "PKV_ROPE_INTERLEAVED",
    "PKV_OK", "PKV_ERR_INVALID_ARG", "PKV_ERR_UNSUPPORTED", "PKV_ERR_WORKSPACE",
    "PKV_ERR_CUDA", "PKV_ERR_BOUNDS", "PKV_ERR_TIMEOUT",
    "PKV_F16", "PKV_BF16", "PKV_FP8_E4M3", "PKV_F32", "PKV_FP8_E4M3_TOKEN", "PKV_STEP_OVERLAP",
    "EXPORTED_SYMBOLS",
]

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE = 0, 1, 2, 3
PKV_ERR_CUDA, PKV_ERR_BOUNDS, PKV_ERR_TIMEOUT = 4, 5, 6
PKV_F16, PKV_BF16, PKV_FP8_E4M3, PKV_F32, PKV_FP8_E4M3_TOKEN = 0, 1, 2, 3, 4
PKV_STEP_OVERLAP = 1
PKV_ROPE_INTERLEAVED = 1
PKV_MAX_TREE = 64

EXPORTED_SYMBOLS = (
    "pkv_kv_append", "pkv_decode_workspace_bytes", "pkv_paged_decode_attention",
    "pkv_decode_step", "pkv_kv_bytes_per_token", "pkv_status_string", "pkv_version",
    "pkv_paged_decode_attention_noalloc", "pkv_copy_blocks", "pkv_paged_decode_attention_multi",
    "pkv_paged_decode_attention_window", "pkv_decode_step_fused", "pkv_paged_prefill_attention",
    "pkv_decode_workspace_bytes_multi", "pkv_kv_append_rope",
    "pkv_paged_decode_attention_biased", "pkv_paged_prefill_attention_biased",
    "pkv_paged_decode_attention_shared_prefix", "pkv_shared_prefix_workspace_bytes",
    "pkv_paged_decode_attention_scored", "pkv_scored_workspace_bytes", "pkv_kv_evict",
    "pkv_paged_tree_attention", "pkv_tree_workspace_bytes", "pkv_kv_accept_path",
)
PKV_NOALLOC_SCRATCH_BYTES = 32 << 20

_DTYPE_CODE = {torch.float16: PKV_F16, torch.bfloat16: PKV_BF16,
               torch.uint8: PKV_FP8_E4M3, torch.float32: PKV_F32}
if hasattr(torch, "float8_e4m3fn"):
    _DTYPE_CODE[torch.float8_e4m3fn] = PKV_FP8_E4M3


class PkvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {pkv_status_string(status)}")


class CacheDesc(ctypes.Structure):
    """Mirror of ``pkv_cache_desc`` (include/pkv.h)."""
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("num_blocks", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("cache_dtype", ctypes.c_int32),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("err_word", ctypes.c_void_p),
    ]


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def load_library():
    """Load libpkv.so (building it with nvcc if absent or stale)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build()
        lib = ctypes.CDLL(path)
        P, I32, U64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t
        D = ctypes.POINTER(CacheDesc)
        lib.pkv_kv_append.restype = I32
        lib.pkv_kv_append.argtypes = [D, P, P, P, P, P, I32, I32, P]
        lib.pkv_decode_workspace_bytes.restype = SZ
        lib.pkv_decode_workspace_bytes.argtypes = [D, I32, I32, I32]
        lib.pkv_decode_workspace_bytes_multi.restype = SZ
        lib.pkv_decode_workspace_bytes_multi.argtypes = [D, I32, I32, I32, I32]
        lib.pkv_paged_decode_attention.restype = I32
        lib.pkv_paged_decode_attention.argtypes = [D, P, P, P, P, P, I32, I32, I32,
                                                   ctypes.c_float, P, I32, I32, P, SZ, P]
        lib.pkv_decode_step.restype = I32
        lib.pkv_decode_step.argtypes = [D, P, P, P, P, P, P, I32, P, P, I32, I32, I32,
                                        ctypes.c_float, P, I32, I32, P, SZ, P]
        lib.pkv_paged_decode_attention_noalloc.restype = I32
        lib.pkv_paged_decode_attention_noalloc.argtypes = [D, P, P, P, P, P, I32, I32, I32,
                                                           ctypes.c_float, P, I32, I32, P]
        lib.pkv_paged_decode_attention_multi.restype = I32
        lib.pkv_paged_decode_attention_multi.argtypes = [D, P, P, P, P, P, I32, I32, I32, I32,
                                                         ctypes.c_float, P, I32, I32, P, SZ, P]
        lib.pkv_paged_prefill_attention.restype = I32
        lib.pkv_paged_prefill_attention.argtypes = [D, P, P, P, P, P, P, I32, I32, I32, I32,
                                                    ctypes.c_float, P, I32, I32, P]
        lib.pkv_decode_step_fused.restype = I32
        lib.pkv_decode_step_fused.argtypes = [D, P, P, P, P, P, I32, P, P, I32, I32, I32,
                                              ctypes.c_float, P, I32, I32, P, SZ, I32, P]
        lib.pkv_paged_decode_attention_window.restype = I32
        lib.pkv_paged_decode_attention_window.argtypes = [D, P, P, P, P, P, I32, I32, I32, I32,
                                                          I32, I32, ctypes.c_float, P, I32, I32,
                                                          P, SZ, P]
        lib.pkv_kv_append_rope.restype = I32
        I64 = ctypes.c_int64
        lib.pkv_kv_append_rope.argtypes = [D, P, P, P, P, P, I32, I32, P, I64, P, I64, P, I64, P,
                                           I32, I32, I32, P]
        F = ctypes.c_float
        lib.pkv_paged_decode_attention_biased.restype = I32
        lib.pkv_paged_decode_attention_biased.argtypes = [D, P, P, P, P, P, I32, I32, I32, F, P,
                                                          I32, I32, F, P, I32, I32, P, SZ, P]
        lib.pkv_paged_prefill_attention_biased.restype = I32
        lib.pkv_paged_prefill_attention_biased.argtypes = [D, P, P, P, P, P, P, I32, I32, I32,
                                                           I32, F, F, P, P, I32, I32, P]
        lib.pkv_shared_prefix_workspace_bytes.restype = SZ
        lib.pkv_shared_prefix_workspace_bytes.argtypes = [D, I32, I32, I32, I32]
        lib.pkv_paged_decode_attention_shared_prefix.restype = I32
        lib.pkv_paged_decode_attention_shared_prefix.argtypes = [D, P, P, P, P, I32, P, P, I32,
                                                                 I32, I32, F, P, I32, I32, P, SZ,
                                                                 P]
        lib.pkv_scored_workspace_bytes.restype = SZ
        lib.pkv_scored_workspace_bytes.argtypes = [D, I32, I32, I32]
        lib.pkv_paged_decode_attention_scored.restype = I32
        lib.pkv_paged_decode_attention_scored.argtypes = [D, P, P, P, P, P, P, F, I32, I32, I32,
                                                          F, P, I32, I32, P, SZ, P]
        lib.pkv_tree_workspace_bytes.restype = SZ
        lib.pkv_tree_workspace_bytes.argtypes = [D, I32, I32, I32]
        lib.pkv_paged_tree_attention.restype = I32
        lib.pkv_paged_tree_attention.argtypes = [D, P, P, P, P, P, P, I32, I32, I32, P, I32, F, P,
                                                 I32, I32, P, SZ, P]
        lib.pkv_kv_accept_path.restype = I32
        lib.pkv_kv_accept_path.argtypes = [D, P, P, P, P, P, P, P, I32, I32, I32, P, P]
        lib.pkv_kv_evict.restype = I32
        lib.pkv_kv_evict.argtypes = [D, P, P, P, P, P, P, P, P, I32, I32, I32, I32, I32, P, P]
        lib.pkv_copy_blocks.restype = I32
        lib.pkv_copy_blocks.argtypes = [D, P, P, P, P, I32, P]
        lib.pkv_kv_bytes_per_token.restype = U64
        lib.pkv_kv_bytes_per_token.argtypes = [I32, I32, I32, I32]
        lib.pkv_status_string.restype = ctypes.c_char_p
        lib.pkv_status_string.argtypes = [I32]
        lib.pkv_version.restype = I32
        lib.pkv_version.argtypes = []
        _lib = lib
        return lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _dev_ptr(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


# The calls below are made every few microseconds by a decode loop: pointers go
# to ctypes as plain ints, and the current device and stream are read without
# building torch objects for them.
def _on(t: Optional[torch.Tensor], dev: int, name: str) -> Optional[int]:
    """Device address of a contiguous tensor on device dev."""
    if t is None:
        return None
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor, on the device of q")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream_on(stream, dev: int) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def _is_current(dev: int) -> bool:
    """Whether dev is the current device (the library works on that one); a host
    tensor's -1 passes, to be named by the check of the tensor."""
    if dev < 0:
        return True
    return dev == (_raw_device() if _raw_device is not None else torch.cuda.current_device())


def _stream_handle(stream, device) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def make_desc(num_blocks: int, page_size: int, num_kv_heads: int, num_q_heads: int,
              head_dim: int, cache_dtype: int, k_scale: Optional[torch.Tensor] = None,
              v_scale: Optional[torch.Tensor] = None,
              err_word: Optional[torch.Tensor] = None) -> CacheDesc:
    """Build a ``pkv_cache_desc``.  Tensors passed here must outlive its use."""
    d = CacheDesc()
    d.struct_size = ctypes.sizeof(CacheDesc)
    d.num_blocks = num_blocks
    d.page_size = page_size
    d.num_kv_heads = num_kv_heads
    d.num_q_heads = num_q_heads
    d.head_dim = head_dim
    d.cache_dtype = cache_dtype
    d.k_scale = k_scale.data_ptr() if k_scale is not None else None
    d.v_scale = v_scale.data_ptr() if v_scale is not None else None
    d.err_word = err_word.data_ptr() if err_word is not None else None
    return d


def _check(status: int, where: str):
    if status != PKV_OK:
        raise PkvError(status, where)


def pkv_kv_append(desc: CacheDesc, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  slot_mapping: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  stream=None) -> None:
    """k, v: [T][Hkv][d] (fp16/bf16); slot_mapping: int64 [T]."""
    lib = load_library()
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must match")
    st = lib.pkv_kv_append(ctypes.byref(desc), _dev_ptr(k_cache, "k_cache"),
                           _dev_ptr(v_cache, "v_cache"), _dev_ptr(slot_mapping, "slot_mapping"),
                           _dev_ptr(k, "k"), _dev_ptr(v, "v"), int(k.shape[0]),
                           _DTYPE_CODE.get(k.dtype, -1), _stream_handle(stream, k.device))
    _check(st, "pkv_kv_append")


def pkv_kv_append_rope(desc: CacheDesc, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       slot_mapping: torch.Tensor, positions: torch.Tensor,
                       cos_sin: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       q_out: torch.Tensor, interleaved: bool = False, stream=None) -> None:
    """q: [T][Hq][d], k, v: [T][Hkv][d] (fp16/bf16), the tokens of each at any
    stride; slot_mapping, positions: int64 [T]; cos_sin: fp32
    [max_position][rot_dim], a position's cosines then its sines; q_out:
    [T][Hq][d], which may be q."""
    lib = _lib or load_library()
    dev = q.get_device()
    if not _is_current(dev):
        with torch.cuda.device(dev):
            return pkv_kv_append_rope(desc, k_cache, v_cache, slot_mapping, positions, cos_sin, q,
                                      k, v, q_out, interleaved, stream)
    i64 = torch.int64
    if slot_mapping.dtype is not i64 or positions.dtype is not i64:
        raise ValueError("slot_mapping and positions must be int64")
    if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be fp32 [max_position][rot_dim]")
    dt = q.dtype
    if k.dtype is not dt or v.dtype is not dt or q_out.dtype is not dt:
        raise ValueError("q, k, v and q_out must have one type")
    T, Hq, Hkv, d = slot_mapping.numel(), desc.num_q_heads, desc.num_kv_heads, desc.head_dim
    if positions.numel() != T:
        raise ValueError("slot_mapping and positions need one entry per token")
    qshape, kvshape = (T, Hq, d), (T, Hkv, d)
    if q.shape != qshape or q_out.shape != qshape or k.shape != kvshape or v.shape != kvshape:
        raise ValueError("q and q_out must be [T][Hq][d], k and v [T][Hkv][d]")
    (qs, qh, qd), (ks, kh, kd), (vs, vh, vd) = q.stride(), k.stride(), v.stride()
    if not (qd == kd == vd == 1 and (qh == d or Hq == 1) and (kh == vh == d or Hkv == 1)):
        raise ValueError("the heads of a token of q, k and v must be contiguous")
    if T == 1:  # the stride of a single row says nothing
        qs, ks, vs = Hq * d, Hkv * d, Hkv * d
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("k and v must be on the device of q")
    max_pos, rot = cos_sin.shape
    st = lib.pkv_kv_append_rope(
        ctypes.byref(desc), _on(k_cache, dev, "k_cache"), _on(v_cache, dev, "v_cache"),
        _on(slot_mapping, dev, "slot_mapping"), _on(positions, dev, "positions"),
        _on(cos_sin, dev, "cos_sin"), max_pos, rot, q.data_ptr(), qs, k.data_ptr(), ks,
        v.data_ptr(), vs, _on(q_out, dev, "q_out"), T, _DTYPE_CODE.get(dt, -1),
        PKV_ROPE_INTERLEAVED if interleaved else 0, _stream_on(stream, dev))
    if st:
        raise PkvError(st, "pkv_kv_append_rope")


def pkv_copy_blocks(desc: CacheDesc, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    src_blocks: torch.Tensor, dst_blocks: torch.Tensor, stream=None) -> None:
    """Block dst_blocks[i] of both caches receives block src_blocks[i] (int32)."""
    lib = load_library()
    if src_blocks.dtype != torch.int32 or dst_blocks.dtype != torch.int32:
        raise ValueError("block ids must be int32")
    if src_blocks.numel() != dst_blocks.numel():
        raise ValueError("src_blocks and dst_blocks must have the same length")
    st = lib.pkv_copy_blocks(ctypes.byref(desc), _dev_ptr(k_cache, "k_cache"),
                             _dev_ptr(v_cache, "v_cache"), _dev_ptr(src_blocks, "src_blocks"),
                             _dev_ptr(dst_blocks, "dst_blocks"), int(src_blocks.numel()),
                             _stream_handle(stream, k_cache.device))
    _check(st, "pkv_copy_blocks")


def pkv_decode_workspace_bytes(desc: CacheDesc, batch: int, max_blocks_per_seq: int,
                               max_context_len_hint: int = 0) -> int:
    lib = load_library()
    return int(lib.pkv_decode_workspace_bytes(ctypes.byref(desc), int(batch),
                                              int(max_blocks_per_seq),
                                              int(max_context_len_hint)))


def pkv_decode_workspace_bytes_multi(desc: CacheDesc, batch: int, q_len: int,
                                     max_blocks_per_seq: int,
                                     max_context_len_hint: int = 0) -> int:
    lib = load_library()
    return int(lib.pkv_decode_workspace_bytes_multi(ctypes.byref(desc), int(batch), int(q_len),
                                                    int(max_blocks_per_seq),
                                                    int(max_context_len_hint)))


def pkv_paged_decode_attention(desc: CacheDesc, q: torch.Tensor, k_cache: torch.Tensor,
                               v_cache: torch.Tensor, block_tables: torch.Tensor,
                               context_lens: torch.Tensor, scale: float, out: torch.Tensor,
                               workspace: torch.Tensor, max_context_len_hint: int = 0,
                               stream=None) -> None:
    """q/out: [B][Hq][d]; block_tables int32 [B][MBS]; context_lens int32 [B]."""
    lib = load_library()
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    B, mbs = int(block_tables.shape[0]), int(block_tables.shape[1])
    st = lib.pkv_paged_decode_attention(
        ctypes.byref(desc), _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"),
        _dev_ptr(v_cache, "v_cache"), _dev_ptr(block_tables, "block_tables"),
        _dev_ptr(context_lens, "context_lens"), B, mbs, int(max_context_len_hint),
        float(scale), _dev_ptr(out, "out"), _DTYPE_CODE.get(q.dtype, -1),
        _DTYPE_CODE.get(out.dtype, -1), _dev_ptr(workspace, "workspace"),
        int(workspace.numel() * workspace.element_size()), _stream_handle(stream, q.device))
    _check(st, "pkv_paged_decode_attention")


def pkv_paged_decode_attention_multi(desc: CacheDesc, q: torch.Tensor, k_cache: torch.Tensor,
                                     v_cache: torch.Tensor, block_tables: torch.Tensor,
                                     context_lens: torch.Tensor, scale: float,
                                     out: torch.Tensor, workspace: torch.Tensor,
                                     max_context_len_hint: int = 0, stream=None) -> None:
    """q/out: [B][q_len][Hq][d], the last q_len tokens of each sequence, causal
    among themselves; block_tables int32 [B][MBS]; context_lens int32 [B]."""
    lib = load_library()
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if q.dim() != 4 or out.shape != q.shape:
        raise ValueError("q and out must be [B][q_len][Hq][d]")
    B, mbs = int(block_tables.shape[0]), int(block_tables.shape[1])
    st = lib.pkv_paged_decode_attention_multi(
        ctypes.byref(desc), _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"),
        _dev_ptr(v_cache, "v_cache"), _dev_ptr(block_tables, "block_tables"),
        _dev_ptr(context_lens, "context_lens"), B, int(q.shape[1]), mbs,
        int(max_context_len_hint), float(scale), _dev_ptr(out, "out"),
        _DTYPE_CODE.get(q.dtype, -1), _DTYPE_CODE.get(out.dtype, -1),
        _dev_ptr(workspace, "workspace"), int(workspace.numel() * workspace.element_size()),
        _stream_handle(stream, q.device))
    _check(st, "pkv_paged_decode_attention_multi")


def pkv_paged_decode_attention_window(desc: CacheDesc, q: torch.Tensor, k_cache: torch.Tensor,
                                      v_cache: torch.Tensor, block_tables: torch.Tensor,
                                      context_lens: torch.Tensor, window: int, sinks: int,
                                      scale: float, out: torch.Tensor, workspace: torch.Tensor,
                                      max_context_len_hint: int = 0, stream=None) -> None:
    """As pkv_paged_decode_attention_multi, token t seeing only positions
    t - window + 1 .. t and the first `sinks` positions (window 0: no window)."""
    lib = load_library()
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if q.dim() != 4 or out.shape != q.shape:
        raise ValueError("q and out must be [B][q_len][Hq][d]")
    B, mbs = int(block_tables.shape[0]), int(block_tables.shape[1])
    st = lib.pkv_paged_decode_attention_window(
        ctypes.byref(desc), _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"),
        _dev_ptr(v_cache, "v_cache"), _dev_ptr(block_tables, "block_tables"),
        _dev_ptr(context_lens, "context_lens"), B, int(q.shape[1]), int(window), int(sinks),
        mbs, int(max_context_len_hint), float(scale), _dev_ptr(out, "out"),
        _DTYPE_CODE.get(q.dtype, -1), _DTYPE_CODE.get(out.dtype, -1),
        _dev_ptr(workspace, "workspace"), int(workspace.numel() * workspace.element_size()),
        _stream_handle(stream, q.device))
    _check(st, "pkv_paged_decode_attention_window")


def _bias_on(alibi_slopes: Optional[torch.Tensor], dev: int, desc: CacheDesc) -> Optional[int]:
    if alibi_slopes is None:
        return None
    if alibi_slopes.dtype != torch.float32 or alibi_slopes.numel() != desc.num_q_heads:
        raise ValueError("alibi_slopes must be fp32 with one entry per query head")
    return _on(alibi_slopes, dev, "alibi_slopes")


def _batch_of(desc: CacheDesc, q: torch.Tensor, out: torch.Tensor, block_tables: torch.Tensor,
              context_lens: torch.Tensor):
    """Batch and table width of a single-token call, its shapes checked."""
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    B, mbs = block_tables.shape
    want = (B, desc.num_q_heads, desc.head_dim)
    if q.shape != want or out.shape != want:
        raise ValueError("q and out must be [B][Hq][d]")
    if context_lens.numel() != B:
        raise ValueError("context_lens needs one entry per sequence")
    return B, mbs


def pkv_paged_decode_attention_biased(desc: CacheDesc, q: torch.Tensor, k_cache: torch.Tensor,
                                      v_cache: torch.Tensor, block_tables: torch.Tensor,
                                      context_lens: torch.Tensor, scale: float,
                                      out: torch.Tensor, workspace: torch.Tensor,
                                      softcap: float = 0.0,
                                      alibi_slopes: Optional[torch.Tensor] = None,
                                      window: int = 0, sinks: int = 0,
                                      max_context_len_hint: int = 0, stream=None) -> None:
    """As pkv_paged_decode_attention, a score s becoming softcap tanh(s /
    softcap) (softcap > 0), then s + alibi_slopes[hq] (u - t) (fp32 [Hq]; key
    position u, query position t); window and sinks as for the windowed call."""
    lib = _lib or load_library()
    dev = q.get_device()
    if not _is_current(dev):
        with torch.cuda.device(dev):
            return pkv_paged_decode_attention_biased(
                desc, q, k_cache, v_cache, block_tables, context_lens, scale, out, workspace,
                softcap, alibi_slopes, window, sinks, max_context_len_hint, stream)
    B, mbs = _batch_of(desc, q, out, block_tables, context_lens)
    st = lib.pkv_paged_decode_attention_biased(
        ctypes.byref(desc), _on(q, dev, "q"), _on(k_cache, dev, "k_cache"),
        _on(v_cache, dev, "v_cache"), _on(block_tables, dev, "block_tables"),
        _on(context_lens, dev, "context_lens"), B, int(window), int(sinks), float(softcap),
        _bias_on(alibi_slopes, dev, desc), mbs, int(max_context_len_hint), float(scale),
        _on(out, dev, "out"), _DTYPE_CODE.get(q.dtype, -1), _DTYPE_CODE.get(out.dtype, -1),
        _on(workspace, dev, "workspace"), workspace.nbytes, _stream_on(stream, dev))
    if st:
        raise PkvError(st, "pkv_paged_decode_attention_biased")


def pkv_scored_workspace_bytes(desc: CacheDesc, batch: int, max_blocks_per_seq: int,
                               max_context_len_hint: int = 0) -> int:
    lib = load_library()
    return int(lib.pkv_scored_workspace_bytes(ctypes.byref(desc), int(batch),
                                              int(max_blocks_per_seq),
                                              int(max_context_len_hint)))


def _row_pool(t: torch.Tensor, dtype, desc: CacheDesc, dev: int, name: str) -> int:
    """Device address of a pool with one entry per cached row."""
    if t.dtype is not dtype or t.numel() != desc.num_blocks * desc.num_kv_heads * desc.page_size:
        raise ValueError(f"{name} must be {dtype} [num_blocks][Hkv][page_size]")
    return _on(t, dev, name)


def pkv_paged_decode_attention_scored(desc: CacheDesc, q: torch.Tensor, k_cache: torch.Tensor,
                                      v_cache: torch.Tensor, block_tables: torch.Tensor,
                                      context_lens: torch.Tensor, weights: torch.Tensor,
                                      scale: float, out: torch.Tensor, workspace: torch.Tensor,
                                      decay: float = 1.0, max_context_len_hint: int = 0,
                                      stream=None) -> None:
    """As pkv_paged_decode_attention; weights (fp32 [num_blocks][Hkv][16]) of the
    rows seen become decay * weights + the attention weight of the KV head's query
    heads, the newest row's (and with decay 0 all of them) the latter alone.  Set the
    weights of other rows that came since the last such call (to 0) before this one."""
    lib = _lib or load_library()
    dev = q.get_device()
    if not _is_current(dev):
        with torch.cuda.device(dev):
            return pkv_paged_decode_attention_scored(
                desc, q, k_cache, v_cache, block_tables, context_lens, weights, scale, out,
                workspace, decay, max_context_len_hint, stream)
    B, mbs = _batch_of(desc, q, out, block_tables, context_lens)
    st = lib.pkv_paged_decode_attention_scored(
        ctypes.byref(desc), _on(q, dev, "q"), _on(k_cache, dev, "k_cache"),
        _on(v_cache, dev, "v_cache"), _on(block_tables, dev, "block_tables"),
        _on(context_lens, dev, "context_lens"),
        _row_pool(weights, torch.float32, desc, dev, "weights"), float(decay), B, mbs,
        int(max_context_len_hint), float(scale), _on(out, dev, "out"),
        _DTYPE_CODE.get(q.dtype, -1), _DTYPE_CODE.get(out.dtype, -1),
        _on(workspace, dev, "workspace"), workspace.nbytes, _stream_on(stream, dev))
    if st:
        raise PkvError(st, "pkv_paged_decode_attention_scored")


def pkv_kv_evict(desc: CacheDesc, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 weights: torch.Tensor, positions: torch.Tensor, block_tables: torch.Tensor,
                 context_lens: torch.Tensor, old_lens: torch.Tensor, num_tokens: torch.Tensor,
                 budget: int, sinks: int, recent: int, new_context_lens: torch.Tensor,
                 stream=None) -> None:
    """Keep `budget` rows of each sequence under each KV head: those of its first
    `sinks` and last `recent` tokens, then those with the largest weights.  weights
    (fp32) and positions (int32: the token of a row) are [num_blocks][Hkv][16];
    context_lens, old_lens (rows whose positions are known), num_tokens (tokens in
    all) and new_context_lens (written) int32 [B]."""
    lib = _lib or load_library()
    dev = k_cache.get_device()
    if not _is_current(dev):
        with torch.cuda.device(dev):
            return pkv_kv_evict(desc, k_cache, v_cache, weights, positions, block_tables,
                                context_lens, old_lens, num_tokens, budget, sinks, recent,
                                new_context_lens, stream)
    i32 = torch.int32
    if (block_tables.dtype is not i32 or context_lens.dtype is not i32
            or old_lens.dtype is not i32 or num_tokens.dtype is not i32
            or new_context_lens.dtype is not i32):
        raise ValueError("block_tables, context_lens, old_lens, num_tokens and "
                         "new_context_lens must be int32")
    B, mbs = block_tables.shape
    if not (context_lens.numel() == old_lens.numel() == num_tokens.numel()
            == new_context_lens.numel() == B):
        raise ValueError("the lengths need one entry per sequence")
    st = lib.pkv_kv_evict(
        ctypes.byref(desc), _on(k_cache, dev, "k_cache"), _on(v_cache, dev, "v_cache"),
        _row_pool(weights, torch.float32, desc, dev, "weights"),
        _row_pool(positions, i32, desc, dev, "positions"), _on(block_tables, dev, "block_tables"),
        _on(context_lens, dev, "context_lens"), _on(old_lens, dev, "old_lens"),
        _on(num_tokens, dev, "num_tokens"), B, mbs, int(budget), int(sinks), int(recent),
        _on(new_context_lens, dev, "new_context_lens"), _stream_on(stream, dev))
    if st:
        raise PkvError(st, "pkv_kv_evict")


def pkv_tree_workspace_bytes(desc: CacheDesc, batch: int, max_q_len: int,
                             max_blocks_per_seq: int) -> int:
    lib = load_library()
    return int(lib.pkv_tree_workspace_bytes(ctypes.byref(desc), int(batch), int(max_q_len),
                                            int(max_blocks_per_seq)))


def pkv_paged_tree_attention(desc: CacheDesc, q: torch.Tensor, k_cache: torch.Tensor,
                             v_cache: torch.Tensor, block_tables: torch.Tensor,
                             context_lens: torch.Tensor, q_start: torch.Tensor, max_q_len: int,
                             tree_mask: torch.Tensor, scale: float, out: torch.Tensor,
                             workspace: torch.Tensor, stream=None) -> None:
    """q/out: [total_q][Hq][d]; sequence b's nodes are rows q_start[b] ..
    q_start[b+1]-1 (at most 64), cached at its last positions.  A node sees every
    position before the tree and node i where bit i of its word in tree_mask (int64
    [total_q]) is set."""
    lib = _lib or load_library()
    dev = q.get_device()
    if not _is_current(dev):
        with torch.cuda.device(dev):
            return pkv_paged_tree_attention(desc, q, k_cache, v_cache, block_tables, context_lens,
                                            q_start, max_q_len, tree_mask, scale, out, workspace,
                                            stream)
    i32 = torch.int32
    if block_tables.dtype is not i32 or context_lens.dtype is not i32 or q_start.dtype is not i32:
        raise ValueError("block_tables, context_lens and q_start must be int32")
    total = q.shape[0]
    want = (total, desc.num_q_heads, desc.head_dim)
    if q.shape != want or out.shape != want:
        raise ValueError("q and out must be [total_q][Hq][d]")
    if tree_mask.dtype is not torch.int64 or tree_mask.numel() != total:
        raise ValueError("tree_mask must be int64 with one word per row of q")
    B, mbs = block_tables.shape
    if q_start.numel() != B + 1 or context_lens.numel() != B:
        raise ValueError("q_start needs batch + 1 entries and context_lens batch")
    st = lib.pkv_paged_tree_attention(
        ctypes.byref(desc), _on(q, dev, "q"), _on(k_cache, dev, "k_cache"),
        _on(v_cache, dev, "v_cache"), _on(block_tables, dev, "block_tables"),
        _on(context_lens, dev, "context_lens"), _on(q_start, dev, "q_start"), B, total,
        int(max_q_len), _on(tree_mask, dev, "tree_mask"), mbs, float(scale),
        _on(out, dev, "out"), _DTYPE_CODE.get(q.dtype, -1), _DTYPE_CODE.get(out.dtype, -1),
        _on(workspace, dev, "workspace"), workspace.nbytes, _stream_on(stream, dev))
    if st:
        raise PkvError(st, "pkv_paged_tree_attention")


def pkv_kv_accept_path(desc: CacheDesc, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       block_tables: torch.Tensor, context_lens: torch.Tensor,
                       q_start: torch.Tensor, path: torch.Tensor, path_lens: torch.Tensor,
                       new_context_lens: Optional[torch.Tensor] = None, stream=None) -> None:
    """The rows of nodes path[b][:path_lens[b]] (int32 [B][max_path]) of each
    sequence's tree move up behind its past, in that order; new_context_lens (int32
    [B], written) counts the past and the path.  Weights and positions of rows (see
    pkv_kv_evict) do not move."""
    lib = _lib or load_library()
    dev = k_cache.get_device()
    if not _is_current(dev):
        with torch.cuda.device(dev):
            return pkv_kv_accept_path(desc, k_cache, v_cache, block_tables, context_lens, q_start,
                                      path, path_lens, new_context_lens, stream)
    i32 = torch.int32
    if (block_tables.dtype is not i32 or context_lens.dtype is not i32
            or q_start.dtype is not i32 or path.dtype is not i32 or path_lens.dtype is not i32):
        raise ValueError("block_tables, context_lens, q_start, path and path_lens must be int32")
    B, mbs = block_tables.shape
    if (q_start.numel() != B + 1 or context_lens.numel() != B or path_lens.numel() != B
            or path.dim() != 2 or path.shape[0] != B):
        raise ValueError("q_start needs batch + 1 entries, context_lens, path and path_lens batch")
    if new_context_lens is not None and (new_context_lens.dtype is not i32
                                         or new_context_lens.numel() != B):
        raise ValueError("new_context_lens must be int32 with one entry per sequence")
    st = lib.pkv_kv_accept_path(
        ctypes.byref(desc), _on(k_cache, dev, "k_cache"), _on(v_cache, dev, "v_cache"),
        _on(block_tables, dev, "block_tables"), _on(context_lens, dev, "context_lens"),
        _on(q_start, dev, "q_start"), _on(path, dev, "path"), _on(path_lens, dev, "path_lens"),
        path.shape[1], B, mbs, _on(new_context_lens, dev, "new_context_lens"),
        _stream_on(stream, dev))
    if st:
        raise PkvError(st, "pkv_kv_accept_path")


def pkv_shared_prefix_workspace_bytes(desc: CacheDesc, batch: int, num_prefix_blocks: int,
                                      max_blocks_per_seq: int,
                                      max_context_len_hint: int = 0) -> int:
    lib = load_library()
    return int(lib.pkv_shared_prefix_workspace_bytes(ctypes.byref(desc), int(batch),
                                                     int(num_prefix_blocks),
                                                     int(max_blocks_per_seq),
                                                     int(max_context_len_hint)))


def pkv_paged_decode_attention_shared_prefix(desc: CacheDesc, q: torch.Tensor,
                                             k_cache: torch.Tensor, v_cache: torch.Tensor,
                                             prefix_blocks: torch.Tensor,
                                             block_tables: torch.Tensor,
                                             context_lens: torch.Tensor, scale: float,
                                             out: torch.Tensor, workspace: torch.Tensor,
                                             max_context_len_hint: int = 0,
                                             stream=None) -> None:
    """As pkv_paged_decode_attention for sequences that all begin with the
    blocks prefix_blocks (int32 [num_prefix_blocks]), which are read once for
    every 256 query rows of a KV head (short prefixes and small batches: once per
    sequence); block_tables holds whole tables, whose entries for the prefix are
    not read, and context_lens whole lengths."""
    lib = _lib or load_library()
    dev = q.get_device()
    if not _is_current(dev):
        with torch.cuda.device(dev):
            return pkv_paged_decode_attention_shared_prefix(
                desc, q, k_cache, v_cache, prefix_blocks, block_tables, context_lens, scale, out,
                workspace, max_context_len_hint, stream)
    if prefix_blocks.dtype != torch.int32:
        raise ValueError("prefix_blocks must be int32")
    B, mbs = _batch_of(desc, q, out, block_tables, context_lens)
    st = lib.pkv_paged_decode_attention_shared_prefix(
        ctypes.byref(desc), _on(q, dev, "q"), _on(k_cache, dev, "k_cache"),
        _on(v_cache, dev, "v_cache"), _on(prefix_blocks, dev, "prefix_blocks"),
        prefix_blocks.numel(), _on(block_tables, dev, "block_tables"),
        _on(context_lens, dev, "context_lens"), B, mbs, int(max_context_len_hint),
        float(scale),
        _on(out, dev, "out"), _DTYPE_CODE.get(q.dtype, -1), _DTYPE_CODE.get(out.dtype, -1),
        _on(workspace, dev, "workspace"), workspace.nbytes, _stream_on(stream, dev))
    if st:
        raise PkvError(st, "pkv_paged_decode_attention_shared_prefix")


def pkv_decode_step(desc: CacheDesc, q: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, slot_mapping: torch.Tensor, k: torch.Tensor,
                    v: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                    scale: float, out: torch.Tensor, workspace: torch.Tensor,
                    max_context_len_hint: int = 0, stream=None) -> None:
    """Append one token per sequence (k, v: [B][Hkv][d]) then attend."""
    lib = load_library()
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    B, mbs = int(block_tables.shape[0]), int(block_tables.shape[1])
    if k.shape[0] != B or v.shape != k.shape or slot_mapping.shape[0] != B:
        raise ValueError("k, v and slot_mapping need one row per sequence")
    st = lib.pkv_decode_step(
        ctypes.byref(desc), _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"),
        _dev_ptr(v_cache, "v_cache"), _dev_ptr(slot_mapping, "slot_mapping"),
        _dev_ptr(k, "k"), _dev_ptr(v, "v"), _DTYPE_CODE.get(k.dtype, -1),
        _dev_ptr(block_tables, "block_tables"), _dev_ptr(context_lens, "context_lens"),
        B, mbs, int(max_context_len_hint), float(scale), _dev_ptr(out, "out"),
        _DTYPE_CODE.get(q.dtype, -1), _DTYPE_CODE.get(out.dtype, -1),
        _dev_ptr(workspace, "workspace"), int(workspace.numel() * workspace.element_size()),
        _stream_handle(stream, q.device))
    _check(st, "pkv_decode_step")


def pkv_paged_prefill_attention(desc: CacheDesc, q: torch.Tensor, k_cache: torch.Tensor,
                                v_cache: torch.Tensor, block_tables: torch.Tensor,
                                context_lens: torch.Tensor, q_start: torch.Tensor,
                                max_q_len: int, scale: float, out: torch.Tensor,
                                stream=None) -> None:
    """q/out: [total_q][Hq][d]; sequence b's rows q_start[b] .. q_start[b+1]-1
    are its last positions, causal; q_start int32 [B+1] on the device."""
    lib = load_library()
    for t, n in ((block_tables, "block_tables"), (context_lens, "context_lens"),
                 (q_start, "q_start")):
        if t.dtype != torch.int32:
            raise ValueError(f"{n} must be int32")
    if q.dim() != 3 or out.shape != q.shape:
        raise ValueError("q and out must be [total_q][Hq][d]")
    B, mbs = int(block_tables.shape[0]), int(block_tables.shape[1])
    if q_start.numel() != B + 1:
        raise ValueError("q_start needs batch + 1 entries")
    st = lib.pkv_paged_prefill_attention(
        ctypes.byref(desc), _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"),
        _dev_ptr(v_cache, "v_cache"), _dev_ptr(block_tables, "block_tables"),
        _dev_ptr(context_lens, "context_lens"), _dev_ptr(q_start, "q_start"), B,
        int(q.shape[0]), int(max_q_len), mbs, float(scale), _dev_ptr(out, "out"),
        _DTYPE_CODE.get(q.dtype, -1), _DTYPE_CODE.get(out.dtype, -1),
        _stream_handle(stream, q.device))
    _check(st, "pkv_paged_prefill_attention")


def pkv_paged_prefill_attention_biased(desc: CacheDesc, q: torch.Tensor, k_cache: torch.Tensor,
                                       v_cache: torch.Tensor, block_tables: torch.Tensor,
                                       context_lens: torch.Tensor, q_start: torch.Tensor,
                                       max_q_len: int, scale: float, out: torch.Tensor,
                                       softcap: float = 0.0,
                                       alibi_slopes: Optional[torch.Tensor] = None,
                                       stream=None) -> None:
    """As pkv_paged_prefill_attention, the scores changed as by
    pkv_paged_decode_attention_biased (t the row's position)."""
    lib = _lib or load_library()
    dev = q.get_device()
    if not _is_current(dev):
        with torch.cuda.device(dev):
            return pkv_paged_prefill_attention_biased(
                desc, q, k_cache, v_cache, block_tables, context_lens, q_start, max_q_len, scale,
                out, softcap, alibi_slopes, stream)
    if (block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32
            or q_start.dtype != torch.int32):
        raise ValueError("block_tables, context_lens and q_start must be int32")
    total = q.shape[0]
    want = (total, desc.num_q_heads, desc.head_dim)
    if q.shape != want or out.shape != want:
        raise ValueError("q and out must be [total_q][Hq][d]")
    B, mbs = block_tables.shape
    if q_start.numel() != B + 1 or context_lens.numel() != B:
        raise ValueError("q_start needs batch + 1 entries and context_lens batch")
    st = lib.pkv_paged_prefill_attention_biased(
        ctypes.byref(desc), _on(q, dev, "q"), _on(k_cache, dev, "k_cache"),
        _on(v_cache, dev, "v_cache"), _on(block_tables, dev, "block_tables"),
        _on(context_lens, dev, "context_lens"), _on(q_start, dev, "q_start"), B, total,
        int(max_q_len), mbs, float(scale), float(softcap), _bias_on(alibi_slopes, dev, desc),
        _on(out, dev, "out"),
        _DTYPE_CODE.get(q.dtype, -1), _DTYPE_CODE.get(out.dtype, -1), _stream_on(stream, dev))
    if st:
        raise PkvError(st, "pkv_paged_prefill_attention_biased")


def pkv_decode_step_fused(desc: CacheDesc, q: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                          out: torch.Tensor, workspace: torch.Tensor,
                          max_context_len_hint: int = 0, stream=None,
                          overlap: bool = False) -> None:
    """One kernel: sequence b's new token (k[b], v[b]: [B][Hkv][d]) goes to its
    position context_lens[b] - 1, then every sequence attends.  overlap sets
    PKV_STEP_OVERLAP: context_lens and block_tables are not written by the
    kernel launched just before on the stream."""
    lib = load_library()
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    B, mbs = int(block_tables.shape[0]), int(block_tables.shape[1])
    if k.shape[0] != B or v.shape != k.shape:
        raise ValueError("k and v need one row per sequence")
    st = lib.pkv_decode_step_fused(
        ctypes.byref(desc), _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"),
        _dev_ptr(v_cache, "v_cache"), _dev_ptr(k, "k"), _dev_ptr(v, "v"),
        _DTYPE_CODE.get(k.dtype, -1), _dev_ptr(block_tables, "block_tables"),
        _dev_ptr(context_lens, "context_lens"), B, mbs, int(max_context_len_hint),
        float(scale), _dev_ptr(out, "out"), _DTYPE_CODE.get(q.dtype, -1),
        _DTYPE_CODE.get(out.dtype, -1), _dev_ptr(workspace, "workspace"),
        int(workspace.numel() * workspace.element_size()), PKV_STEP_OVERLAP if overlap else 0,
        _stream_handle(stream, q.device))
    _check(st, "pkv_decode_step_fused")


def pkv_paged_decode_attention_noalloc(desc: CacheDesc, q: torch.Tensor,
                                       k_cache: torch.Tensor, v_cache: torch.Tensor,
                                       block_tables: torch.Tensor, context_lens: torch.Tensor,
                                       scale: float, out: torch.Tensor,
                                       max_context_len_hint: int = 0, stream=None) -> None:
    """Decode attention on the library's fixed device scratch (no workspace).

    For callers that cannot allocate device memory at call time.  Calls that
    overlap on the GPU share the scratch and race; the first call on a device
    should come before any stream capture."""
    lib = load_library()
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    B, mbs = int(block_tables.shape[0]), int(block_tables.shape[1])
    st = lib.pkv_paged_decode_attention_noalloc(
        ctypes.byref(desc), _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"),
        _dev_ptr(v_cache, "v_cache"), _dev_ptr(block_tables, "block_tables"),
        _dev_ptr(context_lens, "context_lens"), B, mbs, int(max_context_len_hint),
        float(scale), _dev_ptr(out, "out"), _DTYPE_CODE.get(q.dtype, -1),
        _DTYPE_CODE.get(out.dtype, -1), _stream_handle(stream, q.device))
    _check(st, "pkv_paged_decode_attention_noalloc")


def pkv_kv_bytes_per_token(layers: int, kv_heads: int, head_dim: int, elem_bytes: int) -> int:
    return int(load_library().pkv_kv_bytes_per_token(layers, kv_heads, head_dim, elem_bytes))


def pkv_status_string(status: int) -> str:
    return load_library().pkv_status_string(int(status)).decode()


def pkv_version() -> int:
    return int(load_library().pkv_version())


@dataclass
class DecodeBuffers:
    """Zero-filled workspace sized for a launch shape (convenience for callers)."""
    workspace: torch.Tensor

    @staticmethod
    def allocate(desc: CacheDesc, batch: int, max_blocks_per_seq: int,
                 max_context_len_hint: int = 0, device="cuda") -> "DecodeBuffers":
        n = pkv_decode_workspace_bytes(desc, batch, max_blocks_per_seq, max_context_len_hint)
        if n == 0:
            raise PkvError(PKV_ERR_INVALID_ARG, "pkv_decode_workspace_bytes")
        return DecodeBuffers(torch.zeros(n, dtype=torch.uint8, device=device))
