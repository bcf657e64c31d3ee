"""pkv_paged_decode_attention_shared_prefix at batches and prefixes large enough
for the prefix to be a pass of its own (4 sequences or more, 32 MB of prefix not
read again), against the formula in 64 bits on sampled sequences."""
import pytest
import torch

from ops_harness import Paged, check
from test_shared_prefix_gpu import expect, shared, workspace
import paged_kv_cache_250_gb300 as pkv

pytestmark = pytest.mark.gpu


def own_pass(p):
    B = len(p.lens)
    return B >= 4 and (B - 1) * p.prefix * p.Hkv * p.d * 4 >= 32 << 20


def spread(n, lo, hi):
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


CASES = [  # prefix, lens, Hq, Hkv, d, cache, out, sampled sequences
    # shorter than the prefix, empty, at its end, just behind it
    (1040, [0, 5, 16, 17, 1039, 1040, 1041, 1100, 0, 1, 1056, 2000], 8, 8, 128, "bf16", "f32",
     range(12)),
    # nobody reaches the prefix's end: what lies behind 1500 was never written
    (2048, [1500, 3, 1499, 0, 128, 129, 1000, 700], 8, 8, 128, "f16", "f32", range(8)),
    # nobody sees anything
    (2048, [0] * 8, 8, 8, 128, "bf16", "f32", range(8)),
    # 256, 264 and 320 rows of a KV head: a whole pair of tiles, 8 and 64 rows more
    (1040, spread(32, 1041, 1300), 32, 4, 128, "bf16", "f32", [0, 15, 16, 31]),
    (1040, spread(33, 1041, 1300), 32, 4, 128, "bf16", "bf16", [0, 15, 16, 31, 32]),
    (1040, spread(40, 900, 1300), 32, 4, 128, "bf16", "f32", [0, 15, 16, 31, 32, 39]),
    # one query head per KV head
    (1040, spread(20, 1040, 1100), 32, 32, 64, "f16", "f16", [0, 1, 10, 19]),
    # groups of two and four, head dim 64, a prefix that ends inside a block
    (2064, spread(100, 2064, 2200), 4, 2, 64, "bf16", "f32", [0, 63, 64, 99]),
    (4112, spread(64, 4112, 4130), 12, 3, 64, "f16", "f32", [0, 31, 32, 63]),
    # 720 rows: three pairs, the last whole
    (2064, spread(90, 2065, 2100), 16, 2, 128, "bf16", "f32", [0, 31, 32, 63, 64, 89]),
    # long own parts, many chunks each
    (4096, [4097, 9000, 4500, 5000, 4096], 16, 8, 128, "bf16", "f32", range(5)),
]


@pytest.mark.parametrize("case", CASES)
def test_matches_the_formula(case):
    prefix, lens, Hq, Hkv, d, cache, out, rows = case
    p = Paged(lens, Hq, Hkv, d, cache, 71, prefix=prefix)
    assert own_pass(p)
    q = p.queries(len(lens), 72, 2.0)
    ws = workspace(p)
    o = shared(p, q, out, ws=ws)
    assert p.err.item() == 0
    rows = list(rows)
    ref, tol = expect(p, q, rows)
    check(o[rows], ref, tol, out, str(case[:1] + case[2:7]))
    assert torch.isfinite(o).all()
    assert torch.equal(o, shared(p, q, out, ws=ws))
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.all(o[b] == 0)


def test_hints():
    """A hint changes the cut, not the answer; one below the true lengths too."""
    lens = spread(24, 2050, 3500)
    p = Paged(lens, 8, 4, 128, "bf16", 73, prefix=2048)
    assert own_pass(p)
    q = p.queries(24, 74)
    ws = workspace(p)
    rows = [0, 11, 23]
    ref, tol = expect(p, q, rows)
    for hint in (0, 3500, 2100, 17, 10 ** 6):
        check(shared(p, q, ws=ws, hint=hint)[rows], ref, tol, "f32", f"hint {hint}")


def test_one_workspace_for_large_and_small_calls_and_their_graphs():
    big = Paged(spread(64, 2048, 2300), 8, 4, 128, "bf16", 75, prefix=2048)
    mid = Paged(spread(6, 5000, 6000), 8, 4, 128, "bf16", 76, prefix=4992)
    one = Paged([700, 800], 8, 4, 128, "bf16", 77, prefix=640)  # a single kernel
    assert own_pass(big) and own_pass(mid) and not own_pass(one)
    n = max(pkv.pkv_shared_prefix_workspace_bytes(x.desc, 64, 128, 400) for x in (big, mid, one))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    calls = []
    for x in (big, mid, one):
        q = x.queries(len(x.lens), 78)
        rows = sorted({0, 1, len(x.lens) // 2, len(x.lens) - 1})
        want = expect(x, q, rows)
        first = shared(x, q, ws=ws)
        check(first[rows], *want, "f32")
        dq, o = q.cuda(), torch.empty(len(x.lens), 8, 128, device="cuda")
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            pkv.pkv_paged_decode_attention_shared_prefix(
                x.desc, dq, x.kc, x.vc, x.prefix_blocks, x.tables, x.ctx, x.scale, o, ws)
        calls.append((g, o, dq, first))
    for i in (0, 1, 2, 0, 0, 2, 1, 1, 0):
        calls[i][1].fill_(float("nan"))
        calls[i][0].replay()
    torch.cuda.synchronize()
    for g, o, dq, first in calls:
        assert torch.equal(o, first)


def test_back_to_back_calls_do_not_mix():
    """Many calls queued without a wait, on one workspace, with new queries each:
    a call's three kernels overlap one another and the next call's start."""
    p = Paged(spread(48, 2048, 2400), 8, 4, 128, "bf16", 79, prefix=2048)
    assert own_pass(p)
    ws = workspace(p)
    qs = [p.queries(48, 80 + i, 2.0).cuda() for i in range(12)]
    outs = [torch.empty(48, 8, 128, device="cuda") for _ in qs]
    for q, o in zip(qs, outs):
        pkv.pkv_paged_decode_attention_shared_prefix(p.desc, q, p.kc, p.vc, p.prefix_blocks,
                                                     p.tables, p.ctx, p.scale, o, ws)
    torch.cuda.synchronize()
    for q, o in zip(qs, outs):
        assert torch.equal(o, shared(p, q.cpu(), ws=ws))


def test_two_streams_with_a_workspace_each():
    p = Paged(spread(48, 2048, 2400), 8, 4, 128, "bf16", 95, prefix=2048)
    want = []
    qs = [p.queries(48, 96 + i).cuda() for i in range(2)]
    for q in qs:
        want.append(shared(p, q.cpu()))
    wss = [workspace(p) for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [[torch.empty(48, 8, 128, device="cuda") for _ in range(6)] for _ in qs]
    torch.cuda.synchronize()
    for i in range(6):
        for q, ws, st, o in zip(qs, wss, streams, outs):
            pkv.pkv_paged_decode_attention_shared_prefix(p.desc, q, p.kc, p.vc, p.prefix_blocks,
                                                         p.tables, p.ctx, p.scale, o[i], ws,
                                                         stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            assert torch.equal(x, w)


def test_bad_blocks_and_lengths_are_reported():
    p = Paged(spread(48, 2048, 2400), 8, 4, 128, "bf16", 81, prefix=2048)
    assert own_pass(p)
    q = p.queries(48, 82)
    for bad in (-1, p.NB, 2 ** 30):
        good = int(p.prefix_blocks[3])
        p.prefix_blocks[3] = bad
        shared(p, q)
        assert p.err.item() == pkv.PKV_ERR_BOUNDS
        p.err.zero_()
        p.prefix_blocks[3] = good
    good = int(p.tables[40, 130])  # an own page
    p.tables[40, 130] = p.NB + 5
    o = shared(p, q)
    assert p.err.item() == pkv.PKV_ERR_BOUNDS
    rows = [0, 39, 41, 47]
    check(o[rows], *expect(p, q, rows), "f32")
    p.err.zero_()
    p.tables[40, 130] = good
    p.ctx[7] = p.mbs * 16 + 5
    p.ctx[8] = -3
    o = shared(p, q)
    assert p.err.item() == pkv.PKV_ERR_BOUNDS
    assert torch.all(o[7] == 0) and torch.all(o[8] == 0)
    rows = [0, 6, 9, 47]
    check(o[rows], *expect(p, q, rows), "f32")


def test_nan_shows_where_it_is_seen():
    """A NaN in a sequence's own rows reaches that sequence and KV head alone, one
    in a prefix's key every sequence that sees it."""
    p = Paged([2048 + 5 * i for i in range(47)] + [100], 8, 4, 128, "bf16", 83, prefix=2048)
    assert own_pass(p)
    q = p.queries(48, 84)
    page = int(p.tables[5, 129])
    p.kc[page, 1, 2, 0] = float("nan")
    o = shared(p, q)
    assert torch.isnan(o[5, 2:4]).all()
    assert torch.isfinite(o[5, :2]).all() and torch.isfinite(o[5, 4:]).all()
    rows = [0, 4, 6, 47]
    check(o[rows], *expect(p, q, rows), "f32")
    p.kc[int(p.prefix_blocks[100]), 3, 7, 9] = float("nan")
    o = shared(p, q)
    assert torch.isnan(o[:47, 6:]).all() and torch.isfinite(o[47]).all()
    assert torch.isfinite(o[:5, :6]).all()


def test_a_batch_of_thousands():
    """More pairs of row tiles than SMs; own parts of at most a page."""
    B = 3000
    p = Paged([272 + b % 17 for b in range(B)], 16, 2, 64, "f16", 85, prefix=272)
    assert own_pass(p)
    q = p.queries(B, 86)
    o = shared(p, q)
    rows = [0, 1, 17, 1500, 2047, 2048, 2999]
    check(o[rows], *expect(p, q, rows), "f32")
    assert torch.isfinite(o).all()
