"""Attention for trees of drafted tokens against the formula in fp64."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import DT, PAGE, Paged, check

pytestmark = pytest.mark.gpu


def trees(nodes, seed):
    """One word per node: its ancestors' bits and its own, parents drawn."""
    g = torch.Generator().manual_seed(seed)
    words = []
    for n in nodes:
        mine = []
        for j in range(n):
            up = int(torch.randint(0, j + 1, (1,), generator=g)) - 1  # -1: hangs on the past
            mine.append((mine[up] if up >= 0 else 0) | 1 << j)
        words += mine
    return words


def as_int64(words):
    return torch.tensor([w - (1 << 64) if w >> 63 & 1 else w for w in words], dtype=torch.int64)


def starts_of(nodes):
    return torch.tensor([0] + list(torch.tensor(nodes).cumsum(0)), dtype=torch.int32)


def tree(p, q, nodes, words, out_type="f32", ws=None, out=None, most=None, stream=None):
    q = q.cuda()
    if out is None:
        out = torch.full(q.shape, 7.0, dtype=DT[out_type], device="cuda")
    most = most or max(nodes)
    if ws is None:  # it need not be cleared
        n = pkv.pkv_tree_workspace_bytes(p.desc, len(nodes), most, p.mbs)
        ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_tree_attention(p.desc, q, p.kc, p.vc, p.tables, p.ctx,
                                 starts_of(nodes).cuda(), most, as_int64(words).cuda(), p.scale,
                                 out, ws, stream=stream)
    return out


def expect(p, q, nodes, words, gone=()):
    """fp64, with the error the kernel may make: that of ops_harness.attend."""
    ref = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape[:2], dtype=torch.float64)
    r, g = 0, p.Hq // p.Hkv
    for b, n in enumerate(nodes):
        base = p.lens[b] - n
        for j in range(n):
            see = torch.ones(p.lens[b], dtype=torch.bool)
            for i in range(n):
                see[base + i] = words[r] >> i & 1
            for bb, page in gone:
                if bb == b:
                    see[page * PAGE:(page + 1) * PAGE] = False
            u = see.nonzero()[:, 0]
            if len(u):
                for h in range(p.Hkv):
                    k, v = p.K[b][u, h], p.V[b][u, h]
                    x = q[r, h * g:(h + 1) * g].double()
                    s = x @ k.T * p.scale
                    size = (x.abs() @ k.abs().T * p.scale).amax(1)
                    w = torch.exp(s - s.amax(1, keepdim=True))
                    ref[r, h * g:(h + 1) * g] = w @ v / w.sum(1, keepdim=True)
                    ds = size * p.d * 2.0 ** -23
                    tol[r, h * g:(h + 1) * g] = v.abs().max() * 2 * (ds + 2.0 ** -15)
            r += 1
    return ref, tol


SHAPES = [(8, 8, 64, "f16"), (8, 4, 128, "bf16"), (8, 2, 128, "f16"), (8, 1, 64, "bf16"),
          (24, 3, 128, "bf16"), (4, 4, 128, "f16")]


@pytest.mark.parametrize("Hq,Hkv,d,cache", SHAPES)
def test_ragged_trees(Hq, Hkv, d, cache):
    pasts = [0, 1, 15, 16, 17, 127, 128, 129, 0, 300, 64, 700]
    nodes = [1, 64, 3, 16, 33, 1, 7, 0, 31, 64, 65 - 16, 2]
    p = Paged([a + n for a, n in zip(pasts, nodes)], Hq, Hkv, d, cache, 11)
    q = p.queries(sum(nodes), 12, 2.0)
    words = trees(nodes, 13)
    out = tree(p, q, nodes, words)
    check(out, *expect(p, q, nodes, words), "f32")
    assert p.err.item() == 0
    assert torch.equal(out, tree(p, q, nodes, words))


@pytest.mark.parametrize("out_type", ["f16", "bf16", "f32"])
def test_output_types(out_type):
    nodes = [5, 20]
    p = Paged([105, 20], 8, 2, 128, "f16", 21)
    q = p.queries(25, 22, 2.0)
    words = trees(nodes, 23)
    check(tree(p, q, nodes, words, out_type), *expect(p, q, nodes, words), out_type)


@pytest.mark.parametrize("Hq,Hkv,nodes,past", [(8, 1, 64, 5000), (4, 1, 7, 9001), (8, 8, 1, 3333),
                                               (8, 2, 40, 2500)])
def test_one_long_sequence_is_split(Hq, Hkv, nodes, past):
    p = Paged([past + nodes], Hq, Hkv, 128, "bf16", 31)
    q = p.queries(nodes, 32, 3.0)
    words = trees([nodes], 33)
    check(tree(p, q, [nodes], words), *expect(p, q, [nodes], words), "f32")


def test_a_chain_is_the_multi_query_call():
    B, n = 6, 8
    p = Paged([40, 8, 300, 129, 17, 1000], 8, 2, 128, "bf16", 41)
    q = p.queries(B * n, 42, 2.0)
    out = tree(p, q, [n] * B, [(2 << j) - 1 for j in range(n)] * B)
    ws = torch.zeros(pkv.pkv_decode_workspace_bytes_multi(p.desc, B, n, p.mbs), dtype=torch.uint8,
                     device="cuda")
    want = torch.empty(B, n, 8, 128, device="cuda")
    pkv.pkv_paged_decode_attention_multi(p.desc, q.view(B, n, 8, 128).cuda(), p.kc, p.vc, p.tables,
                                         p.ctx, p.scale, want, ws)
    # both carry the weights as pairs of 16-bit values: 2^-15 of the values each
    bound = 2 * 2.0 ** -14 * max(v.abs().max() for v in p.V)
    assert (out.view_as(want) - want).abs().max() <= bound


def test_any_mask_and_rows_that_see_nothing():
    """Masks need not be trees; bits past the tree are ignored; a row without any
    position is zero."""
    nodes = [64, 10, 10, 1, 1]
    p = Paged([64, 10, 150, 1, 20], 8, 2, 128, "f16", 51)
    g = torch.Generator().manual_seed(52)
    words = [int(torch.randint(0, 2, (1,), generator=g)) for _ in range(sum(nodes))]
    words = [sum(int(torch.randint(0, 2, (1,), generator=g)) << i for i in range(64))
             for _ in words]
    words[3], words[63] = 0, 1 << 63
    words[64 + 2], words[64 + 3] = 0, (1 << 64) - (1 << 10)
    words[64 + 10 + 5] = 0
    words[-2] = 0
    q = p.queries(sum(nodes), 53, 2.0)
    out = tree(p, q, nodes, words)
    ref, tol = expect(p, q, nodes, words)
    check(out, ref, tol, "f32")
    for r in (3, 64 + 2, 64 + 3, -2):
        assert torch.all(out[r] == 0)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("Hq", [4, 16])
def test_a_node_that_nobody_sees_may_hold_anything(value, Hq):
    nodes, lens = [30, 64], [200, 64]
    p = Paged(lens, Hq, 2, 128, "bf16", 61)
    words = trees(nodes, 62)
    for b, i in ((0, 0), (0, 17), (0, 29), (1, 5), (1, 63)):
        u = lens[b] - nodes[b] + i
        blk = int(p.tables[b, u // PAGE])
        p.kc[blk, :, u % PAGE] = value
        p.vc[blk, :, u % PAGE] = value
        at = sum(nodes[:b])
        for j in range(nodes[b]):
            words[at + j] &= ~(1 << i)
    q = p.queries(sum(nodes), 63, 2.0)
    check(tree(p, q, nodes, words), *expect(p, q, nodes, words), "f32")


def test_masked_keys_may_hold_anything():
    """A node whose key is NaN for those that do not see it: only its own row shows it."""
    nodes, lens = [12], [140]
    p = Paged(lens, 8, 2, 64, "f16", 71)
    words = trees(nodes, 72)
    for j in range(12):
        words[j] &= ~(1 << 4)
    words[4] |= 1 << 4
    u = 128 + 4
    p.kc[int(p.tables[0, u // PAGE]), :, u % PAGE] = float("nan")
    q = p.queries(12, 73, 2.0)
    out = tree(p, q, nodes, words)
    assert torch.isnan(out[4]).all()
    ref, tol = expect(p, q, nodes, words)
    others = [j for j in range(12) if j != 4]
    check(out[others], ref[others], tol[others], "f32")


def test_bad_counts_leave_their_rows_alone():
    nodes = [5, 9, 6, 0, 8]
    for bad in ("count", "short", "long", "negative"):
        p = Paged([50, 90, 60, 4, 80], 8, 2, 128, "bf16", 81)
        words = trees(nodes, 82)
        q = p.queries(sum(nodes) + 3, 83, 2.0)
        ctx = p.ctx.clone()
        most = 9
        if bad == "count":
            most = 8
        elif bad == "short":
            ctx[1] = 8
        elif bad == "long":
            ctx[1] = p.mbs * PAGE + 1
        else:
            ctx[1] = -1
        p.ctx = ctx
        out = tree(p, q, nodes, words + [1, 1, 1], most=most)
        ref, tol = expect(p, q[:28], nodes, words)
        good = list(range(5)) + list(range(14, 28))
        check(out[good], ref[good], tol[good], "f32")
        assert torch.all(out[5:14] == 7.0) and torch.all(out[28:] == 7.0)
        assert p.err.item() == pkv.PKV_ERR_BOUNDS


def test_starts_that_run_backwards_or_past_the_rows():
    p = Paged([50, 60], 8, 2, 128, "bf16", 91)
    q = p.queries(10, 92).cuda()
    ws = torch.zeros(pkv.pkv_tree_workspace_bytes(p.desc, 2, 8, p.mbs), dtype=torch.uint8,
                     device="cuda")
    mask = torch.full((10,), 3, dtype=torch.int64, device="cuda")
    for starts in ([0, 6, 12], [4, 2, 5], [-2, 3, 6], [9, 17, 9]):
        p.err.zero_()
        out = torch.full(q.shape, 7.0, device="cuda")
        pkv.pkv_paged_tree_attention(p.desc, q, p.kc, p.vc, p.tables, p.ctx,
                                     torch.tensor(starts, dtype=torch.int32).cuda(), 8, mask,
                                     p.scale, out, ws)
        assert p.err.item() == pkv.PKV_ERR_BOUNDS, starts
        for b in range(2):
            a, z = starts[b], starts[b + 1]
            if 0 <= a <= z <= 10:
                assert torch.isfinite(out[a:z]).all() and not (out[a:z] == 7.0).all()


@pytest.mark.parametrize("Hq", [2, 16])
def test_blocks_outside_the_pool_are_left_out(Hq):
    nodes, lens = [9, 40], [400, 300]
    p = Paged(lens, Hq, 2, 128, "f16", 101)
    gone = [(0, 3), (0, 24), (1, 0), (1, 17)]
    for i, (b, page) in enumerate(gone):
        p.tables[b, page] = (-1, p.NB, 1 << 30, -(1 << 31))[i]
    words = trees(nodes, 102)
    q = p.queries(sum(nodes), 103, 2.0)
    out = tree(p, q, nodes, words)
    check(out, *expect(p, q, nodes, words, gone), "f32")
    assert p.err.item() == pkv.PKV_ERR_BOUNDS


def test_hundreds_of_small_trees():
    g = torch.Generator().manual_seed(111)
    nodes = torch.randint(0, 9, (400,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(nodes, torch.randint(0, 150, (400,), generator=g))]
    p = Paged(lens, 4, 2, 64, "bf16", 112)
    words = trees(nodes, 113)
    q = p.queries(sum(nodes), 114, 2.0)
    check(tree(p, q, nodes, words), *expect(p, q, nodes, words), "f32")


def test_one_workspace_for_graphs_of_large_and_small_calls():
    runs = []
    big = Paged([900 + 7 * i for i in range(9)], 8, 2, 128, "bf16", 121)
    small = Paged([77], 8, 2, 128, "bf16", 122)
    size = max(pkv.pkv_tree_workspace_bytes(p.desc, len(p.lens), 64, p.mbs) for p in (big, small))
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    for p, nodes in ((big, [30 + i for i in range(9)]), (small, [11])):
        words = trees(nodes, 123)
        qs = [p.queries(sum(nodes), 124 + i, 2.0) for i in range(2)]
        want = [tree(p, q, nodes, words) for q in qs]
        check(want[1], *expect(p, qs[1], nodes, words), "f32")
        dq, o = qs[0].cuda(), torch.empty_like(want[0])
        st, mask = starts_of(nodes).cuda(), as_int64(words).cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pkv.pkv_paged_tree_attention(p.desc, dq, p.kc, p.vc, p.tables, p.ctx, st, 64, mask,
                                         p.scale, o, ws)
        runs.append((g, dq, o, qs, want, st, mask))
    for i, which in ((0, 0), (1, 0), (0, 1), (1, 1), (1, 0), (0, 0)):
        g, dq, o, qs, want = runs[i][:5]
        dq.copy_(qs[which])
        o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[which])


def test_two_streams_with_a_workspace_each():
    nodes = [20] * 12
    p = Paged([1500 + 50 * i for i in range(12)], 8, 2, 128, "bf16", 131)
    words = trees(nodes, 132)
    qs = [p.queries(240, 133 + i, 2.0) for i in range(2)]
    want = [tree(p, q, nodes, words) for q in qs]
    n = pkv.pkv_tree_workspace_bytes(p.desc, 12, 20, p.mbs)
    wss = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    dqs = [q.cuda() for q in qs]
    outs = [[torch.empty_like(want[0]) for _ in range(6)] for _ in qs]
    mask, st = as_int64(words).cuda(), starts_of(nodes).cuda()
    torch.cuda.synchronize()
    for i in range(6):
        for q, ws, s, o in zip(dqs, wss, streams, outs):
            pkv.pkv_paged_tree_attention(p.desc, q, p.kc, p.vc, p.tables, p.ctx, st, 20, mask,
                                         p.scale, o[i], ws, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            assert torch.equal(x, w)


def test_the_largest_batch():
    """More sequences than the kernel keeps at hand, some of them empty or alone."""
    g = torch.Generator().manual_seed(141)
    B = 3328
    nodes = torch.randint(0, 4, (B,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(nodes, torch.randint(0, 20, (B,), generator=g))]
    p = Paged(lens, 2, 1, 64, "f16", 142)
    words = trees(nodes, 143)
    q = p.queries(sum(nodes), 144, 2.0)
    check(tree(p, q, nodes, words), *expect(p, q, nodes, words), "f32")
    assert p.err.item() == 0


def test_a_graph_whose_trees_and_lengths_change():
    """Segments of one tile and of two, cut and whole, from one captured call."""
    cap = [2500, 900, 300, 64]
    p = Paged(cap, 16, 2, 128, "bf16", 151)
    q = p.queries(200, 152, 2.0)
    dq, o = q.cuda(), torch.empty(200, 16, 128, device="cuda")
    starts = torch.zeros(5, dtype=torch.int32, device="cuda")
    mask = torch.zeros(200, dtype=torch.int64, device="cuda")
    ws = torch.full((pkv.pkv_tree_workspace_bytes(p.desc, 4, 64, p.mbs),), 0xff,
                    dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pkv.pkv_paged_tree_attention(p.desc, dq, p.kc, p.vc, p.tables, p.ctx, starts, 64, mask,
                                     p.scale, o, ws)
    K, V = p.K, p.V
    for i, (nodes, lens) in enumerate([([64, 64, 64, 8], cap), ([3, 0, 17, 64], [2500, 5, 17, 64]),
                                       ([16, 16, 16, 16], [16, 900, 129, 30]),
                                       ([0, 0, 0, 1], [0, 1, 2, 1]), ([64, 1, 64, 1], cap)]):
        words = trees(nodes, 153 + i)
        n = sum(nodes)
        p.ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        starts.copy_(starts_of(nodes))
        mask[:n] = as_int64(words).cuda()
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        p.lens = lens
        p.K, p.V = [k[:x] for k, x in zip(K, lens)], [v[:x] for v, x in zip(V, lens)]
        ref, tol = expect(p, q[:n], nodes, words)
        check(o[:n], ref, tol, "f32")
        assert torch.all(o[n:] == 7.0)
    assert p.err.item() == 0
