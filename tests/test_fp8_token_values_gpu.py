"""Per-token E4M3 caches whose V rows are far from unit size: a row's scale goes into
its softmax weight before the product with V, and has to keep the weight's bits there.
The rows' codes are as drawn; their scales are multiplied by powers of two, so the
references stay exact."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import PAGE, Paged, attend, check

pytestmark = pytest.mark.gpu

LENS = [1, 15, 33, 64, 200, 1023, 5000, 0, 17]


def scaled(Hq, Hkv, size, seed, lens=LENS):
    """V rows of 2^size, or of 2^-20 to 2^20 each."""
    p = Paged(lens, Hq, Hkv, 128, "e4m3tok", seed)
    g = torch.Generator().manual_seed(seed + 1)
    ks = p.ks.cpu()
    for b, n in enumerate(lens):
        e = torch.randint(-20, 21, (n, Hkv), generator=g) if size == "mixed" else \
            torch.full((n, Hkv), size)
        up = torch.exp2(e.double())
        u = torch.arange(n)
        blk, off = p.tables[b].cpu().long()[u // PAGE], u % PAGE
        ks[blk, :, 1, off] *= up.float()
        p.V[b] = p.V[b] * up[..., None]
    p.ks.copy_(ks)
    return p


def expect(p, q, at=lambda b, j: 0):
    """q [B][rows][Hq][d]; row j of sequence b sees all but its last at(b, j) tokens."""
    ref, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape[:3]).double()
    for b, n in enumerate(p.lens):
        for j in range(q.shape[1]):
            ref[b, j], tol[b, j] = attend(q[b, j].double(), p.K[b], p.V[b], p.scale,
                                          n - 1 - at(b, j))
    return ref, tol


SIZES = [-30, -10, -7, -3, 0, 12, 60, "mixed"]


def compare(p, out, ref, tol):
    check(out, ref, tol, "f32")
    assert p.err.item() == 0


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (16, 2)])
def test_decode_plain_and_scored(size, Hq, Hkv):
    p = scaled(Hq, Hkv, size, 11)
    B = len(LENS)
    q = p.queries(B, 12, 2.0)
    ref, tol = expect(p, q[:, None])
    out = torch.empty(q.shape, device="cuda")
    ws = zeros(pkv.pkv_decode_workspace_bytes(p.desc, B, p.mbs))
    pkv.pkv_paged_decode_attention(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, p.scale, out, ws)
    compare(p, out, ref[:, 0], tol[:, 0])
    ws = zeros(pkv.pkv_scored_workspace_bytes(p.desc, B, p.mbs))
    weights = torch.zeros(p.NB, Hkv, PAGE, device="cuda")
    again = torch.empty_like(out)
    pkv.pkv_paged_decode_attention_scored(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, weights,
                                          p.scale, again, ws, decay=0.0)
    compare(p, again, ref[:, 0], tol[:, 0])


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("batch", [3, 110])
def test_both_rings(size, batch):
    """The deep ring and the other one (110 sequences)."""
    lens = ([1200, 40, 333] * batch)[:batch]
    p = scaled(8, 2, size, 21, lens)
    q = p.queries(batch, 22, 2.0)
    out = torch.empty(q.shape, device="cuda")
    ws = zeros(pkv.pkv_decode_workspace_bytes(p.desc, batch, p.mbs))
    pkv.pkv_paged_decode_attention(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, p.scale, out, ws)
    for b in list(range(3)) + [batch - 1]:
        ref, tol = attend(q[b].double(), p.K[b], p.V[b], p.scale, lens[b] - 1)
        compare(p, out[b], ref, tol)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("Hq,Hkv,q_len", [(2, 2, 2), (8, 2, 3), (8, 1, 8)])
def test_multi_query(size, Hq, Hkv, q_len):
    lens = [n for n in LENS if n >= 8]
    p = scaled(Hq, Hkv, size, 31, lens)
    B = len(lens)
    q = p.queries(B * q_len, 32, 2.0).view(B, q_len, Hq, 128)
    out = torch.empty(q.shape, device="cuda")
    ws = zeros(pkv.pkv_decode_workspace_bytes_multi(p.desc, B, q_len, p.mbs))
    pkv.pkv_paged_decode_attention_multi(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, p.scale,
                                         out, ws)
    compare(p, out, *expect(p, q, lambda b, j: q_len - 1 - j))


@pytest.mark.parametrize("size", [-10, "mixed"])
def test_window_and_biased(size):
    p = scaled(8, 2, size, 41)
    B = len(LENS)
    q = p.queries(B, 42, 2.0)
    ws = zeros(pkv.pkv_decode_workspace_bytes(p.desc, B, p.mbs))
    for cap, window, sinks in ((0.0, 100, 4), (30.0, 0, 0), (30.0, 50, 20)):
        out = torch.empty(q.shape, device="cuda")
        pkv.pkv_paged_decode_attention_biased(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx,
                                              p.scale, out, ws, softcap=cap, window=window,
                                              sinks=sinks)
        for b, n in enumerate(LENS):
            ref, tol = attend(q[b].double(), p.K[b], p.V[b], p.scale, n - 1, cap, None, window,
                              sinks)
            compare(p, out[b], ref, tol)


def test_rows_of_zeros_and_what_must_show():
    """Scales of zero (rows of zeros), then an infinite and a NaN scale of a seen row."""
    p = scaled(8, 2, 0, 51, [300, 40])
    q = p.queries(2, 52, 2.0)
    ws = zeros(pkv.pkv_decode_workspace_bytes(p.desc, 2, p.mbs))
    out = torch.empty(q.shape, device="cuda")

    def run():
        pkv.pkv_paged_decode_attention(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, p.scale, out,
                                       ws)
    keep = p.ks.clone()
    p.ks[:, :, 1] = 0.0
    run()
    assert torch.all(out == 0)
    for value in (float("inf"), float("nan")):
        p.ks.copy_(keep)
        p.ks[int(p.tables[0, 5]), 1, 1, 3] = value
        run()
        assert not torch.isfinite(out[0, 4:]).any()
        assert torch.isfinite(out[0, :4]).all() and torch.isfinite(out[1]).all()


def zeros(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")
