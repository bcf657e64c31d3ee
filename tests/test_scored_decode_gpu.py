"""Decode attention that adds up the weight each cached row receives, against the
formula in fp64."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import DT, PAGE, Paged, check

pytestmark = pytest.mark.gpu


def pool_of(p, value=float("nan")):
    return torch.full((p.NB, p.Hkv, PAGE), value, device="cuda")


def workspace(p, B=None, mbs=None):
    n = pkv.pkv_scored_workspace_bytes(p.desc, B or len(p.lens), mbs or p.mbs)
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def scored(p, q, weights, decay=1.0, out_type="f32", ws=None, stream=None):
    out = torch.empty(q.shape, dtype=DT[out_type], device="cuda")
    pkv.pkv_paged_decode_attention_scored(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, weights,
                                          p.scale, out, workspace(p) if ws is None else ws,
                                          decay=decay, stream=stream)
    return out


def expect(p, q, weights, decay, gone=()):
    """Outputs, weights and what the kernel may be off by.

    A score is off by ds (ops_harness.attend), a weight exp(s - lse) by twice that
    relative to itself, 2^-20 for the exponential and the logarithm, and n 2^-24
    for a sum of n terms in any order; adding it up rounds at most twice."""
    g = p.Hq // p.Hkv
    ref, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape[:2]).double()
    w = weights.double().cpu().clone()
    wt = torch.zeros_like(w)
    for b, n in enumerate(p.lens):
        u = torch.tensor([i for i in range(n) if (b, i // PAGE) not in gone], dtype=torch.long)
        if not len(u):
            continue
        blk, off = p.tables[b].cpu().long()[u // PAGE], u % PAGE
        for h in range(p.Hkv):
            k, v = p.K[b][u, h], p.V[b][u, h]
            x = q[b, h * g:(h + 1) * g].double()
            s = x @ k.T * p.scale
            ds = (x.abs() @ k.abs().T * p.scale).amax(1) * p.d * 2.0 ** -23
            pr = torch.softmax(s, 1)
            ref[b, h * g:(h + 1) * g] = pr @ v
            tol[b, h * g:(h + 1) * g] = v.abs().max() * 2 * (ds + 2.0 ** -15)
            old = w[blk, h, off] * decay if decay else torch.zeros(len(u), dtype=torch.float64)
            old[u == n - 1] = 0.0
            w[blk, h, off] = old + pr.sum(0)
            wt[blk, h, off] = (pr * (2 * ds[:, None] + 2.0 ** -20 + n * 2.0 ** -24)).sum(0) + \
                2.0 ** -23 * w[blk, h, off].abs() + 1e-37
    return ref, tol, w, wt


def check_weights(got, w, wt):
    got = got.double().cpu()
    untouched = wt == 0
    assert torch.equal(torch.nan_to_num(got[untouched], -1.0), torch.nan_to_num(w[untouched], -1.0))
    off = (got - w).abs()[~untouched]
    assert (off <= wt[~untouched]).all(), (off / wt[~untouched]).max()


LENS = [1, 15, 16, 17, 0, 64, 200, 1023, 33]


@pytest.mark.parametrize("cache,Hq,Hkv,d", [
    ("f16", 4, 4, 64), ("bf16", 8, 4, 128), ("f16", 8, 2, 128), ("bf16", 16, 2, 64),
    ("e4m3", 4, 4, 128), ("e4m3", 8, 2, 128), ("e4m3tok", 6, 3, 128), ("e4m3tok", 16, 2, 128)])
def test_steps(cache, Hq, Hkv, d):
    """The first step (decay 0) sets every weight, whatever was there; later ones add."""
    p = Paged(LENS, Hq, Hkv, d, cache, 11)
    got, ws = pool_of(p), workspace(p)
    for i, decay in enumerate((0.0, 1.0, 0.75)):
        q = p.queries(len(LENS), 12 + i, 2.0)
        ref, tol, w, wt = expect(p, q, got, decay)
        out = scored(p, q, got, decay, ws=ws)
        check(out, ref, tol, "f32")
        check_weights(got, w, wt)
    assert p.err.item() == 0
    held = torch.isfinite(got).sum().item()
    assert held == Hkv * sum(LENS)  # the others are as they were


def test_outputs_are_those_of_the_plain_call():
    p = Paged([5000, 3, 700, 129], 8, 2, 128, "bf16", 21)
    q = p.queries(4, 22, 2.0)
    for t in ("f16", "bf16", "f32"):
        out = scored(p, q, pool_of(p, 0.0), out_type=t)
        ref, tol, _, _ = expect(p, q, pool_of(p, 0.0), 1.0)
        check(out, ref, tol, t)


@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, 20011), (8, 1, 9000), (32, 32, 701)])
def test_one_sequence_over_many_ctas(Hq, Hkv, n):
    p = Paged([n], Hq, Hkv, 128, "bf16", 31)
    q = p.queries(1, 32, 3.0)
    weights = pool_of(p, 0.5)
    ref, tol, w, wt = expect(p, q, weights, 0.9)
    out = scored(p, q, weights, 0.9)
    check(out, ref, tol, "f32")
    check_weights(weights, w, wt)
    # every head hands out a weight of one
    again = pool_of(p, 0.0)
    scored(p, q, again, 0.0)
    got = again.double().sum((0, 2))
    assert (got - Hq // Hkv).abs().max() <= Hq // Hkv * n * 2.0 ** -22


def test_the_newest_row_starts_from_nothing():
    p = Paged([50, 64], 8, 2, 128, "f16", 41)
    weights = pool_of(p, 3.0)
    for b, n in enumerate(p.lens):
        weights[int(p.tables[b, (n - 1) // PAGE]), :, (n - 1) % PAGE] = float("nan")
    q = p.queries(2, 42)
    scored(p, q, weights)
    for b, n in enumerate(p.lens):
        x = weights[int(p.tables[b, (n - 1) // PAGE]), :, (n - 1) % PAGE]
        assert torch.isfinite(x).all() and (x < 3).all()


def test_blocks_outside_the_pool_are_left_out():
    p = Paged([400, 300, 16], 8, 2, 128, "bf16", 51)
    p.tables[0, 3], p.tables[1, 18], p.tables[2, 0] = -1, p.NB, 1 << 30
    gone = {(0, 3), (1, 18), (2, 0)}
    q = p.queries(3, 52, 2.0)
    weights = pool_of(p, 0.25)
    ref, tol, w, wt = expect(p, q, weights, 1.0, gone)
    out = scored(p, q, weights)
    check(out[:2], ref[:2], tol[:2], "f32")
    assert torch.all(out[2] == 0)
    check_weights(weights, w, wt)
    assert p.err.item() == pkv.PKV_ERR_BOUNDS


def test_lengths_out_of_range_change_no_weight():
    p = Paged([40, 50], 8, 2, 128, "bf16", 61)
    for bad in (-1, p.mbs * PAGE + 1):
        p.ctx[0] = bad
        p.err.zero_()
        weights = pool_of(p, 0.5)
        out = scored(p, p.queries(2, 62), weights)
        assert torch.all(out[0] == 0) and p.err.item() == pkv.PKV_ERR_BOUNDS
        for page in range(3):
            assert torch.all(weights[int(p.tables[0, page])] == 0.5)


def test_nan_shows():
    p = Paged([100], 8, 2, 128, "bf16", 71)
    p.kc[int(p.tables[0, 2]), 1, 3] = float("nan")
    weights = pool_of(p, 0.0)
    out = scored(p, p.queries(1, 72), weights)
    assert torch.isnan(out[0, 4:]).all() and torch.isfinite(out[0, :4]).all()
    blocks = p.tables[0, :7].long()
    assert torch.isnan(weights[blocks, 1].reshape(-1)[:100]).all()
    assert torch.isfinite(weights[blocks, 0].reshape(-1)[:100]).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3tok"])
def test_graphs_of_large_and_small_calls_share_a_workspace(cache):
    big = Paged([3000, 700, 1, 0, 33] * 3, 8, 2, 128, cache, 81)
    small = Paged([900, 17], 8, 2, 128, cache, 82)
    ws = torch.zeros(pkv.pkv_scored_workspace_bytes(big.desc, 15, big.mbs), dtype=torch.uint8,
                     device="cuda")
    runs = []
    for p in (big, small):
        qs = [p.queries(len(p.lens), 83 + i, 2.0) for i in range(2)]
        want = []
        for q in qs:
            w = pool_of(p, 0.125)
            want.append((scored(p, q, w), w))
        dq, o, w = qs[0].cuda(), torch.empty_like(want[0][0]), pool_of(p, 0.125)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pkv.pkv_paged_decode_attention_scored(p.desc, dq, p.kc, p.vc, p.tables, p.ctx, w,
                                                  p.scale, o, ws)
        runs.append((g, dq, o, w, qs, want))
    for i, which in ((0, 0), (1, 0), (0, 1), (1, 1), (1, 0), (0, 0), (0, 1)):
        g, dq, o, w, qs, want = runs[i]
        dq.copy_(qs[which])
        o.fill_(float("nan"))
        w.fill_(0.125)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[which][0]) and torch.equal(w, want[which][1])


def test_two_streams_and_calls_queued_without_a_wait():
    p = Paged([2000 + 50 * i for i in range(12)], 8, 2, 128, "bf16", 91)
    q = p.queries(12, 92, 2.0)
    want_w = pool_of(p, 0.0)
    want = [scored(p, q, want_w, 0.5).clone() for _ in range(5)][-1]
    dq = q.cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [(workspace(p), pool_of(p, 0.0), torch.empty_like(want)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for (ws, w, o), st in zip(sets, streams):
            pkv.pkv_paged_decode_attention_scored(p.desc, dq, p.kc, p.vc, p.tables, p.ctx, w,
                                                  p.scale, o, ws, decay=0.5, stream=st)
    torch.cuda.synchronize()
    for _, w, o in sets:
        assert torch.equal(o, want) and torch.equal(w, want_w)
