"""pkv_paged_decode_attention_shared_prefix against the formula in 64 bits."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import DT, Paged, attend, check

pytestmark = pytest.mark.gpu


def workspace(p, batch=None):
    n = pkv.pkv_shared_prefix_workspace_bytes(p.desc, batch or len(p.lens), p.prefix // 16, p.mbs)
    assert n > 0
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def shared(p, q, out="f32", ws=None, hint=0, stream=None):
    o = torch.full((len(p.lens), p.Hq, p.d), float("nan"), dtype=DT[out], device="cuda")
    pkv.pkv_paged_decode_attention_shared_prefix(
        p.desc, q.cuda(), p.kc, p.vc, p.prefix_blocks, p.tables, p.ctx, p.scale, o,
        workspace(p) if ws is None else ws, max_context_len_hint=hint, stream=stream)
    torch.cuda.synchronize()
    return o


def expect(p, q, rows=None):
    rows = range(len(p.lens)) if rows is None else rows
    r = [attend(q[b].double(), p.K[b], p.V[b], p.scale, p.lens[b] - 1) for b in rows]
    return torch.stack([x[0] for x in r]), torch.stack([x[1] for x in r])


CASES = [  # prefix tokens, lens, Hq, Hkv, d, cache, out
    (64, [65, 64, 70, 81], 8, 2, 128, "bf16", "f32"),
    (16, [17, 300], 4, 4, 64, "f16", "f16"),
    (128, [129, 0, 5, 16, 128, 127, 400], 8, 1, 128, "f16", "f32"),     # shorter than the prefix
    (1040, [1041 + 7 * i for i in range(5)], 8, 8, 64, "f16", "f16"),
    (2064, [2064 + 3 * i for i in range(33)], 8, 2, 64, "bf16", "bf16"),  # 132 rows: a tile and 4
    (272, [273 + i for i in range(40)], 8, 1, 128, "bf16", "f32"),      # 320 rows: two pairs
    (512, [513 + i % 20 for i in range(70)], 8, 2, 128, "bf16", "f32"),   # 280 rows
    (4096, [4100, 4096], 2, 1, 128, "bf16", "f32"),
    (0, [5, 17, 0], 4, 2, 128, "bf16", "f32"),
    (96, [100], 4, 2, 128, "bf16", "f32"),
    (640, [3, 40, 9], 4, 2, 128, "bf16", "f32"),  # nobody reaches the prefix's end
    (64, [0, 0], 4, 2, 64, "f16", "f32"),
]


@pytest.mark.parametrize("case", CASES)
def test_matches_the_formula(case):
    prefix, lens, Hq, Hkv, d, cache, out = case
    p = Paged(lens, Hq, Hkv, d, cache, 51, prefix=prefix)
    q = p.queries(len(lens), 52)
    o = shared(p, q, out)
    assert p.err.item() == 0
    ref, tol = expect(p, q)
    check(o, ref, tol, out, str(case))


def test_many_sequences_sampled_and_repeatable():
    lens = [3000 + (7 * i) % 90 for i in range(150)]
    p = Paged(lens, 16, 2, 128, "bf16", 53, prefix=2992)
    q = p.queries(150, 54, 3.0)
    ws = workspace(p)
    o = shared(p, q, ws=ws)
    rows = [0, 1, 31, 32, 63, 64, 100, 149]
    ref, tol = expect(p, q, rows)
    check(o[rows], ref, tol, "f32")
    for hint in (0, max(lens), 0):
        assert torch.equal(o, shared(p, q, ws=ws, hint=hint))


def test_agrees_with_the_plain_decode():
    """Whole tables: the plain call's answer, to its own accuracy."""
    lens = [700 + i for i in range(48)]
    p = Paged(lens, 8, 2, 128, "bf16", 55, prefix=640, garbage_prefix=False)
    q = p.queries(48, 56)
    ws = torch.zeros(pkv.pkv_decode_workspace_bytes(p.desc, 48, p.mbs), dtype=torch.uint8,
                     device="cuda")
    b = torch.empty(48, 8, 128, device="cuda")
    pkv.pkv_paged_decode_attention(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, p.scale, b, ws)
    ref, tol = expect(p, q)
    check(b, ref, tol, "f32")
    check(shared(p, q), ref, tol, "f32")


def test_workspace_serves_smaller_calls_and_graphs():
    """One workspace: a large batch, a small one, and two captured graphs of
    both, replayed in turn."""
    big = Paged([520 + i for i in range(64)], 8, 2, 128, "bf16", 57, prefix=512)
    small = Paged([2100, 2049, 2080], 8, 2, 128, "bf16", 58, prefix=2048)
    n = max(pkv.pkv_shared_prefix_workspace_bytes(x.desc, 64, 128, 140) for x in (big, small))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    qs = [big.queries(64, 59), small.queries(3, 60)]
    want = [expect(x, q) for x, q in zip((big, small), qs)]
    outs, graphs = [], []
    st = torch.cuda.Stream()
    for x, q in zip((big, small), qs):
        check(shared(x, q, ws=ws), *want[len(outs)], "f32")
        dq = q.cuda()
        o = torch.empty(len(x.lens), 8, 128, device="cuda")
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            pkv.pkv_paged_decode_attention_shared_prefix(
                x.desc, dq, x.kc, x.vc, x.prefix_blocks, x.tables, x.ctx, x.scale, o, ws)
        outs.append((o, dq))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        outs[i][0].fill_(float("nan"))
        graphs[i].replay()
        torch.cuda.synchronize()
        check(outs[i][0], *want[i], "f32")


def test_back_to_back_calls_do_not_mix():
    """Calls queued one behind another on one workspace, each step's new row
    appended in between: the passes of one call overlap one another, not the
    next call's."""
    p = Paged([560 + i for i in range(32)], 8, 2, 128, "bf16", 61, prefix=512)
    ws = workspace(p)
    qs = [p.queries(32, 70 + i).cuda() for i in range(6)]
    outs = [torch.empty(32, 8, 128, device="cuda") for _ in qs]
    for q, o in zip(qs, outs):
        pkv.pkv_paged_decode_attention_shared_prefix(p.desc, q, p.kc, p.vc, p.prefix_blocks,
                                                     p.tables, p.ctx, p.scale, o, ws)
    torch.cuda.synchronize()
    for q, o in zip(qs, outs):
        assert torch.equal(o, shared(p, q.cpu(), ws=ws))


def test_bad_prefix_blocks_and_lengths_are_reported():
    p = Paged([300 + i for i in range(40)], 8, 2, 128, "bf16", 63, prefix=256)
    q = p.queries(40, 64)
    for bad in (-1, p.NB, 2 ** 30):
        good = int(p.prefix_blocks[3])
        p.prefix_blocks[3] = bad
        shared(p, q)
        assert p.err.item() == pkv.PKV_ERR_BOUNDS
        p.err.zero_()
        p.prefix_blocks[3] = good
    p.ctx[7] = p.mbs * 16 + 5
    p.ctx[8] = -3
    o = shared(p, q)
    assert p.err.item() == pkv.PKV_ERR_BOUNDS
    assert torch.all(o[7] == 0) and torch.all(o[8] == 0)
    rows = [0, 6, 9, 39]
    check(o[rows], *expect(p, q, rows), "f32")


def test_nan_shows_where_it_is_seen():
    """A NaN in a sequence's own rows reaches that sequence alone."""
    p = Paged([300 + i for i in range(40)], 8, 2, 128, "bf16", 65, prefix=256)
    q = p.queries(40, 66)
    page = int(p.tables[5, 17])
    p.kc[page, 1, 2, 0] = float("nan")
    o = shared(p, q)
    assert torch.isnan(o[5, 4:]).all() and torch.isfinite(o[5, :4]).all()
    rows = [0, 4, 6, 39]
    check(o[rows], *expect(p, q, rows), "f32")
