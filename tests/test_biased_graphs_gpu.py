"""The biased attention calls captured into graphs: on a side stream, one workspace
for the graphs of several calls, inputs that change between replays."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import Paged, alibi, check
from test_biased_attention_gpu import decode, expect_decode, prefill

pytestmark = pytest.mark.gpu


def captured(call):
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    return g


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e4m3tok"])
def test_decode_graphs_that_share_a_workspace(cache):
    """Capped, biased and plain calls of a large and a small batch, replayed in any
    order: the bits of the same calls made one by one."""
    big = Paged([3000, 700, 1, 0, 33] * 3, 8, 2, 128, cache, 121)
    small = Paged([900, 17], 8, 2, 128, cache, 122)
    n = pkv.pkv_decode_workspace_bytes(big.desc, 15, big.mbs)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    runs = []
    for p, cap, slopes, window in ((big, 30.0, None, 0), (small, 0.0, alibi(8), 0),
                                   (big, 20.0, alibi(8), 100), (small, 0.0, None, 0)):
        B = len(p.lens)
        q, q2 = p.queries(B, 123, 3.0), p.queries(B, 124, 3.0)
        want = [decode(p, x, "f32", cap, slopes, window, ws=ws) for x in (q, q2)]
        ref = expect_decode(p, q2, cap, slopes, window)
        check(want[1], *ref, "f32")
        dq, o = q.cuda(), torch.empty_like(want[0])
        sl = None if slopes is None else slopes.cuda()
        g = captured(lambda: pkv.pkv_paged_decode_attention_biased(
            p.desc, dq, p.kc, p.vc, p.tables, p.ctx, p.scale, o, ws, softcap=cap,
            alibi_slopes=sl, window=window))
        runs.append((g, dq, o, (q, q2), want, sl))
    for i, which in ((0, 0), (1, 0), (2, 0), (3, 0), (1, 1), (0, 1), (3, 1), (2, 1), (0, 0), (1, 0)):
        g, dq, o, qs, want, _ = runs[i]
        dq.copy_(qs[which])
        o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[which])


def test_prefill_in_a_graph_whose_chunks_change():
    p = Paged([400, 333, 64], 8, 2, 128, "bf16", 125)
    sl = alibi(8)
    q = p.queries(300, 126, 3.0)
    dq, dsl = q.cuda(), sl.cuda()
    start = torch.zeros(4, dtype=torch.int32, device="cuda")
    o = torch.full(q.shape, 7.0, device="cuda")
    g = captured(lambda: pkv.pkv_paged_prefill_attention_biased(
        p.desc, dq, p.kc, p.vc, p.tables, p.ctx, start, 200, p.scale, o, softcap=30.0,
        alibi_slopes=dsl))
    for chunks in ([200, 40, 60], [1, 1, 1], [0, 200, 64], [130, 0, 0]):
        start.copy_(torch.tensor([0] + list(torch.tensor(chunks).cumsum(0)), dtype=torch.int32))
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, prefill(p, q, chunks, "f32", 30.0, sl))
        assert torch.all(o[sum(chunks):] == 7.0)
    assert p.err.item() == 0


def test_two_streams_with_a_workspace_each():
    p = Paged([2000 + 50 * i for i in range(12)], 8, 2, 128, "bf16", 127)
    qs = [p.queries(12, 128 + i, 3.0) for i in range(2)]
    want = [decode(p, q, "f32", 30.0) for q in qs]
    dqs = [q.cuda() for q in qs]
    n = pkv.pkv_decode_workspace_bytes(p.desc, 12, p.mbs)
    wss = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [[torch.empty_like(want[0]) for _ in range(8)] for _ in qs]
    torch.cuda.synchronize()
    for i in range(8):
        for q, ws, st, o in zip(dqs, wss, streams, outs):
            pkv.pkv_paged_decode_attention_biased(p.desc, q, p.kc, p.vc, p.tables, p.ctx, p.scale,
                                                  o[i], ws, softcap=30.0, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            assert torch.equal(x, w)
