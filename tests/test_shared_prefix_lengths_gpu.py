"""pkv_paged_decode_attention_shared_prefix where the prefix is a pass of its own
and every sequence ends before the prefix does: the work is cut from the longest
stretch that is seen, the launch is sized from the whole prefix."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import Paged, attend, check
from test_shared_prefix_gpu import expect, shared, workspace
from test_shared_prefix_passes_gpu import own_pass

pytestmark = pytest.mark.gpu


def blocks_over(m, tiles, Hkv):
    """Blocks of 128 tokens with just more than m units of work (a block of a KV
    head and two tiles of rows; half of one with one tile) per SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = 1
    while Hkv * n * tiles // 2 <= m * sms:
        n += 1
    return n


def shape(tiles):  # B, Hq, Hkv: 48 rows of a KV head, or 160
    return (6, 64, 8) if tiles == 1 else (40, 32, 8)


def lengths(B, longest):
    """Two long sequences among short and empty ones."""
    few = [longest, 5, 0, 129, longest - 1, 16]
    return (few + [1 + 7 * i % 90 for i in range(B)])[:B]


@pytest.mark.parametrize("tiles", [1, 2])
@pytest.mark.parametrize("m", [1, 2, 3, 4])
@pytest.mark.parametrize("short", [1, 3])
def test_nobody_reaches_the_end(tiles, m, short):
    """`short` blocks of 128 tokens before it; on a fresh workspace, and on one
    that a call with whole lengths has filled with NaN."""
    B, Hq, Hkv = shape(tiles)
    n = blocks_over(m, tiles, Hkv)
    p = Paged(lengths(B, 128 * (n - short)), Hq, Hkv, 64, "bf16", 101, prefix=128 * n)
    assert own_pass(p)
    q = p.queries(B, 102, 2.0)
    rows = range(6)
    ref, tol = expect(p, q, rows)
    o = shared(p, q)
    check(o[:6], ref, tol, "f32", "fresh")
    assert p.err.item() == 0 and torch.isfinite(o).all()
    ws = workspace(p)
    p.ctx.fill_(128 * n)  # what lies behind the lengths is NaN: so are all partials
    assert torch.isnan(shared(p, q, ws=ws)).all()
    p.ctx.copy_(torch.tensor(p.lens, dtype=torch.int32))
    again = shared(p, q, ws=ws)
    check(again[:6], ref, tol, "f32", "used")
    assert torch.equal(o, again)


def test_lengths_that_shrink_and_grow_under_a_graph():
    """One captured step, replayed with every longest length around the sizes at
    which the cut changes."""
    B, Hq, Hkv = shape(1)
    n = blocks_over(2, 1, Hkv)
    steps = blocks_over(1, 1, Hkv)
    p = Paged([128 * n + 9] * B, Hq, Hkv, 64, "bf16", 105, prefix=128 * n)
    assert own_pass(p)
    q = p.queries(B, 106, 2.0)
    ws, dq = workspace(p), q.cuda()
    o = torch.empty(B, Hq, 64, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        pkv.pkv_paged_decode_attention_shared_prefix(p.desc, dq, p.kc, p.vc, p.prefix_blocks,
                                                     p.tables, p.ctx, p.scale, o, ws)
    for longest in (128 * n + 9, 128 * (n - 1), 128 * steps, 128 * (steps - 1), 1, 0, 128 * n):
        lens = [min(x, longest) for x in lengths(B, max(longest, 1))]
        p.ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(o).all()
        for b in (0, 1, 4):
            t = lens[b] - 1
            ref, tol = attend(q[b].double(), p.K[b], p.V[b], p.scale, t)
            check(o[b], ref, tol, "f32", f"longest {longest}, sequence {b}")
    assert p.err.item() == 0
