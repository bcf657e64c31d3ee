"""What tree attention, path acceptance, scored decode and eviction refuse, on the
host, before any CUDA call."""
import ctypes

import pytest
import torch

import paged_kv_cache_250_gb300 as pkv

F = ctypes.c_void_p(0x10000)   # never dereferenced: validation fails first
N = ctypes.c_void_p(0x90000)   # an array of its own
ODD = ctypes.c_void_p(0x10002)
INV, UNS, WS = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED, pkv.PKV_ERR_WORKSPACE


def desc(Hq=8, Hkv=2, d=128, dtype=pkv.PKV_BF16, page=16):
    x = pkv.make_desc(64, page, Hkv, Hq, d, dtype)
    if dtype in (pkv.PKV_FP8_E4M3, pkv.PKV_FP8_E4M3_TOKEN):
        x.k_scale = x.v_scale = 0x1000
    return x


def tree(x=None, q=F, kc=F, vc=F, tab=F, ctx=F, starts=F, B=2, total=8, most=4, mask=F, mbs=4,
         scale=1.0, out=F, qt=pkv.PKV_BF16, ot=pkv.PKV_F32):
    return pkv.load_library().pkv_paged_tree_attention(
        ctypes.byref(x or desc()), q, kc, vc, tab, ctx, starts, B, total, most, mask, mbs, scale,
        out, qt, ot, F, 1 << 30, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INV), (dict(kc=None), INV), (dict(vc=None), INV), (dict(tab=None), INV),
    (dict(ctx=None), INV), (dict(starts=None), INV), (dict(mask=None), INV), (dict(out=None), INV),
    (dict(q=ODD), INV), (dict(kc=ODD), INV), (dict(out=ODD), INV), (dict(tab=ODD), INV),
    (dict(mask=ctypes.c_void_p(0x10004)), INV), (dict(starts=ODD), INV),
    (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(B=-1), INV), (dict(total=-1), INV),
    (dict(most=-1), INV), (dict(most=65), UNS), (dict(mbs=0), INV), (dict(B=3329), UNS),
    (dict(qt=pkv.PKV_F16), INV), (dict(ot=pkv.PKV_FP8_E4M3), UNS),
    (dict(x=desc(dtype=pkv.PKV_FP8_E4M3)), UNS), (dict(x=desc(dtype=pkv.PKV_FP8_E4M3_TOKEN)), UNS),
    (dict(x=desc(d=96)), UNS), (dict(x=desc(page=32)), UNS), (dict(x=desc(Hq=6)), UNS),
    (dict(B=0, q=None), pkv.PKV_OK), (dict(total=0, q=None), pkv.PKV_OK),
    (dict(most=0, mask=None), pkv.PKV_OK),
])
def test_tree(kw, want):
    assert tree(**kw) == want


def accept(x=None, kc=F, vc=F, tab=F, ctx=F, starts=F, path=F, lens=F, width=4, B=2, mbs=4, new=N):
    return pkv.load_library().pkv_kv_accept_path(
        ctypes.byref(x or desc()), kc, vc, tab, ctx, starts, path, lens, width, B, mbs, new, None)


@pytest.mark.parametrize("kw,want", [
    (dict(kc=None), INV), (dict(vc=None), INV), (dict(tab=None), INV), (dict(ctx=None), INV),
    (dict(starts=None), INV), (dict(path=None), INV), (dict(lens=None), INV), (dict(kc=ODD), INV),
    (dict(path=ODD), INV), (dict(new=ODD), INV), (dict(width=-1), INV), (dict(width=65), UNS),
    (dict(B=-1), INV), (dict(mbs=0), INV), (dict(x=desc(d=96)), UNS), (dict(new=F), INV),
    (dict(new=ctypes.c_void_p(0x10004)), INV),  # overlaps the lengths by one entry
    (dict(B=0, kc=None), pkv.PKV_OK),
])
def test_accept(kw, want):
    assert accept(**kw) == want


def scored(x=None, q=F, kc=F, tab=F, ctx=F, w=F, decay=1.0, B=2, mbs=4, scale=1.0, out=F,
           qt=pkv.PKV_BF16, ot=pkv.PKV_F32, ws=F, n=1 << 30):
    return pkv.load_library().pkv_paged_decode_attention_scored(
        ctypes.byref(x or desc()), q, kc, F, tab, ctx, w, decay, B, mbs, 0, scale, out, qt, ot, ws,
        n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(w=None), INV), (dict(w=ODD), INV), (dict(q=None), INV), (dict(q=ODD), INV),
    (dict(kc=None), INV), (dict(decay=-0.1), INV), (dict(decay=1.1), INV),
    (dict(decay=float("nan")), INV), (dict(scale=float("nan")), INV), (dict(B=-1), INV),
    (dict(mbs=0), INV), (dict(ot=pkv.PKV_FP8_E4M3), UNS), (dict(x=desc(d=96)), UNS),
    (dict(B=7000), UNS), (dict(qt=pkv.PKV_F16), INV),
    (dict(B=0, q=None, w=None, ws=None, n=0), pkv.PKV_OK),
])
def test_scored(kw, want):
    assert scored(**kw) == want


def evict(x=None, kc=F, vc=F, w=F, pos=F, tab=F, ctx=F, old=F, told=F, B=2, mbs=4, budget=8,
          sinks=2, recent=3, new=N):
    return pkv.load_library().pkv_kv_evict(
        ctypes.byref(x or desc()), kc, vc, w, pos, tab, ctx, old, told, B, mbs, budget, sinks,
        recent, new, None)


@pytest.mark.parametrize("kw,want", [
    (dict(kc=None), INV), (dict(vc=None), INV), (dict(w=None), INV), (dict(pos=None), INV),
    (dict(tab=None), INV), (dict(ctx=None), INV), (dict(old=None), INV), (dict(told=None), INV),
    (dict(new=None), INV), (dict(w=ODD), INV), (dict(pos=ODD), INV), (dict(kc=ODD), INV),
    (dict(new=ODD), INV), (dict(budget=0), INV), (dict(budget=-1), INV), (dict(sinks=-1), INV),
    (dict(recent=-1), INV), (dict(sinks=6, recent=3), INV),
    (dict(budget=2 ** 31 - 1, sinks=2 ** 31 - 1, recent=2 ** 31 - 1), INV),
    (dict(B=-1), INV), (dict(mbs=0), INV), (dict(mbs=49153), UNS), (dict(x=desc(d=96)), UNS),
    (dict(new=F), INV), (dict(new=ctypes.c_void_p(0x10000 - 4)), INV),
    (dict(B=0, kc=None), pkv.PKV_OK),
])
def test_evict(kw, want):
    assert evict(**kw) == want


def test_workspace_sizes_of_bad_arguments():
    assert pkv.pkv_tree_workspace_bytes(desc(dtype=pkv.PKV_FP8_E4M3), 2, 4, 8) == 0
    for a in ((0, 4, 8), (2, 0, 8), (2, 65, 8), (2, 4, 0), (-1, 4, 8)):
        assert pkv.pkv_tree_workspace_bytes(desc(), *a) == 0
    for a in ((0, 8), (2, 0), (-1, 8)):
        assert pkv.pkv_scored_workspace_bytes(desc(), *a) == 0


def test_the_binding_checks_types_and_shapes():
    """Host tensors: the binding's own checks come first, then the device's."""
    x = desc()
    i32, i64 = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    q, kc, ws = torch.zeros(3, 8, 128).bfloat16(), torch.zeros(1), torch.zeros(16).byte()
    t, st = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    w, pos = torch.zeros(64, 2, 16), torch.zeros(64, 2, 16, dtype=torch.int32)

    def trees(q=q, t=t, ctx=i32, st=st, mask=i64, out=q):
        pkv.pkv_paged_tree_attention(x, q, kc, kc, t, ctx, st, 1, mask, 1.0, out, ws)
    for kw in (dict(t=t.long()), dict(ctx=i64), dict(st=i32), dict(mask=i32), dict(mask=i64[:2]),
               dict(q=q[:2]), dict(out=q[:, :4]), dict(ctx=i32[:2]), dict()):
        with pytest.raises(ValueError):
            trees(**kw)

    def accepts(t=t, ctx=i32, st=st, path=t, lens=i32, new=None):
        pkv.pkv_kv_accept_path(x, kc, kc, t, ctx, st, path, lens, new)
    for kw in (dict(path=t.long()), dict(path=i32), dict(path=t[:2]), dict(lens=i32[:2]),
               dict(st=i32), dict(new=i64), dict(new=st), dict()):
        with pytest.raises(ValueError):
            accepts(**kw)

    def scores(w=w, q=q, t=t, ctx=i32):
        pkv.pkv_paged_decode_attention_scored(x, q, kc, kc, t, ctx, w, 1.0, q, ws)
    for kw in (dict(w=w.double()), dict(w=w[:63]), dict(q=q[:2]), dict(ctx=i64), dict()):
        with pytest.raises(ValueError):
            scores(**kw)

    def evicts(w=w, pos=pos, t=t, ctx=i32, old=i32, told=i32, new=i32):
        pkv.pkv_kv_evict(x, kc, kc, w, pos, t, ctx, old, told, 8, 1, 1, new)
    for kw in (dict(w=w.half()), dict(pos=pos.long()), dict(pos=pos[:1]), dict(old=i64),
               dict(told=st), dict(new=st), dict(t=t.long()), dict()):
        with pytest.raises(ValueError):
            evicts(**kw)
