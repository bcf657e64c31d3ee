"""What the rotary append, the shared-prefix decode and the biased attention
calls refuse, on the host, before any CUDA call."""
import ctypes

import pytest
import torch

import paged_kv_cache_250_gb300 as pkv

F = ctypes.c_void_p(0x1000)   # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1004)
INV, UNS = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED


def desc(Hq=8, Hkv=2, d=128, dtype=pkv.PKV_BF16):
    x = pkv.make_desc(64, 16, Hkv, Hq, d, dtype)
    if dtype in (pkv.PKV_FP8_E4M3, pkv.PKV_FP8_E4M3_TOKEN):
        x.k_scale = x.v_scale = 0x1000
    return x


def rope(x=None, kc=F, slots=F, pos=F, cs=F, max_pos=10, rot=128, q=F, qs=1024, k=F, ks=256, v=F,
         vs=256, out=F, T=3, dtype=pkv.PKV_BF16, flags=0):
    return pkv.load_library().pkv_kv_append_rope(
        ctypes.byref(x or desc()), kc, F, slots, pos, cs, max_pos, rot, q, qs, k, ks, v, vs, out,
        T, dtype, flags, None)


@pytest.mark.parametrize("kw,want", [
    (dict(kc=None), INV), (dict(slots=None), INV), (dict(pos=None), INV), (dict(cs=None), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(out=None), INV),
    (dict(q=ODD), INV), (dict(out=ODD), INV), (dict(cs=ODD), INV), (dict(pos=ODD), INV),
    (dict(rot=0), INV), (dict(rot=-16), INV), (dict(rot=144), INV), (dict(rot=24), UNS),
    (dict(max_pos=0), INV), (dict(T=-1), INV), (dict(flags=2), INV),
    (dict(qs=1016), INV), (dict(qs=1028), INV), (dict(ks=255), INV), (dict(vs=0), INV),
    (dict(dtype=pkv.PKV_F16), INV), (dict(dtype=pkv.PKV_F32), UNS),
    (dict(x=desc(d=80)), UNS), (dict(T=0, q=None, k=None), pkv.PKV_OK),
])
def test_rope_append(kw, want):
    assert rope(**kw) == want


def biased(x=None, window=0, sinks=0, cap=30.0, slopes=F, q=F, scale=1.0, B=2, ws=F, n=1 << 30,
           out_dtype=pkv.PKV_F32):
    return pkv.load_library().pkv_paged_decode_attention_biased(
        ctypes.byref(x or desc()), q, F, F, F, F, B, window, sinks, cap, slopes, 4, 0, scale, F,
        pkv.PKV_BF16, out_dtype, ws, n, None)


BAD_CAPS = [-1.0, float("nan"), float("inf"), 2.0 ** -11, 2.0 ** 11]


@pytest.mark.parametrize("kw,want", [(dict(cap=c), INV) for c in BAD_CAPS] + [
    (dict(window=-1), INV), (dict(sinks=-1), INV), (dict(slopes=ctypes.c_void_p(0x1001)), INV),
    (dict(q=None), INV), (dict(q=ODD), INV), (dict(scale=float("nan")), INV), (dict(B=-1), INV),
    (dict(out_dtype=pkv.PKV_FP8_E4M3), UNS), (dict(x=desc(d=96)), UNS),
    (dict(x=desc(Hq=48, Hkv=3)), UNS), (dict(B=7000), UNS), (dict(B=0, q=None), pkv.PKV_OK),
])
def test_biased_decode(kw, want):
    assert biased(**kw) == want


def prefill(x=None, cap=30.0, slopes=F, q=F, scale=1.0, B=2, total=8, maxq=4,
            q_dtype=pkv.PKV_BF16):
    return pkv.load_library().pkv_paged_prefill_attention_biased(
        ctypes.byref(x or desc()), q, F, F, F, F, F, B, total, maxq, 4, scale, cap, slopes, F,
        q_dtype, pkv.PKV_F32, None)


@pytest.mark.parametrize("kw,want", [(dict(cap=c), INV) for c in BAD_CAPS] + [
    (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(q=ODD), INV), (dict(total=-1), INV),
    (dict(x=desc(dtype=pkv.PKV_FP8_E4M3)), UNS), (dict(q_dtype=pkv.PKV_F16), INV),
    (dict(B=0), pkv.PKV_OK), (dict(maxq=0), pkv.PKV_OK),
])
def test_biased_prefill(kw, want):
    assert prefill(**kw) == want


def shared(x=None, prefix=F, npb=2, q=F, scale=1.0, B=2, ws=F, n=1 << 30, mbs=4,
           out_dtype=pkv.PKV_F32):
    return pkv.load_library().pkv_paged_decode_attention_shared_prefix(
        ctypes.byref(x or desc()), q, F, F, prefix, npb, F, F, B, mbs, 0, scale, F, pkv.PKV_BF16,
        out_dtype, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(prefix=None), INV), (dict(prefix=ctypes.c_void_p(0x1002)), INV), (dict(npb=-1), INV),
    (dict(npb=5), INV), (dict(scale=0.0), INV), (dict(scale=float("nan")), INV),
    (dict(q=None), INV), (dict(q=ODD), INV), (dict(x=desc(dtype=pkv.PKV_FP8_E4M3)), UNS),
    (dict(x=desc(dtype=pkv.PKV_FP8_E4M3_TOKEN)), UNS), (dict(mbs=0, npb=0), INV),
    (dict(B=7000), UNS), (dict(out_dtype=pkv.PKV_FP8_E4M3), UNS),
    (dict(B=0, q=None, prefix=None, ws=None, n=0), pkv.PKV_OK),
])
def test_shared_prefix(kw, want):
    assert shared(**kw) == want


def test_shared_prefix_workspace_sizes():
    size = pkv.pkv_shared_prefix_workspace_bytes
    assert size(desc(dtype=pkv.PKV_FP8_E4M3), 4, 2, 8) == 0
    assert size(desc(), 4, 9, 8) == 0
    assert size(desc(), 4, -1, 8) == 0
    assert size(desc(), -1, 2, 8) == 0


def test_the_binding_checks_types_and_shapes():
    """Host tensors: the binding's own checks come first, then the device's."""
    x = desc()
    i64, i32 = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    q, k = torch.zeros(3, 8, 128).bfloat16(), torch.zeros(3, 2, 128).bfloat16()
    cs = torch.zeros(10, 128)
    kc = torch.zeros(1)

    def go(slots=i64, pos=i64, cs=cs, q=q, k=k, v=k, out=q):
        pkv.pkv_kv_append_rope(x, kc, kc, slots, pos, cs, q, k, v, out)
    for kw in (dict(slots=i32), dict(pos=i32), dict(cs=cs.double()), dict(cs=cs[0]),
               dict(q=q.half()), dict(v=k.half()), dict(out=q.float()), dict(k=k[:2]),
               dict(q=q[:, :4], out=q[:, :4]), dict(slots=i64[:2]), dict(pos=i64[:2]), dict()):
        with pytest.raises(ValueError):
            go(**kw)
    t = torch.zeros(3, 4, dtype=torch.int32)
    ws = torch.zeros(16, dtype=torch.uint8)
    for kw in (dict(alibi_slopes=torch.zeros(7)), dict(alibi_slopes=torch.zeros(8).double()),
               dict()):
        with pytest.raises(ValueError):
            pkv.pkv_paged_decode_attention_biased(x, q, kc, kc, t, i32, 1.0, q, ws, **kw)
        with pytest.raises(ValueError):
            pkv.pkv_paged_prefill_attention_biased(x, q, kc, kc, t, i32,
                                                   torch.zeros(4, dtype=torch.int32), 1, 1.0, q,
                                                   **kw)
    with pytest.raises(ValueError):
        pkv.pkv_paged_decode_attention_shared_prefix(x, q, kc, kc, i64, t, i32, 1.0, q, ws)
    with pytest.raises(ValueError):
        pkv.pkv_paged_decode_attention_shared_prefix(x, q[:2], kc, kc, i32, t, i32, 1.0, q[:2], ws)
    with pytest.raises(ValueError):
        pkv.pkv_paged_decode_attention_shared_prefix(x, q, kc, kc, i32, t, i32, 1.0, q, ws)
