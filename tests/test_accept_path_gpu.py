"""Acceptance of a path through a tree: whole pools, byte for byte."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import PAGE, Paged

pytestmark = pytest.mark.gpu


def bytes_of(t):
    return t.contiguous().view(torch.uint8)


def spot(p, b, u):
    return int(p.tables[b, u // PAGE]), u % PAGE


def expect(p, nodes, paths):
    kc, vc = p.kc.clone(), p.vc.clone()
    ks = None if p.cache != "e4m3tok" else p.ks.clone()
    for b, (n, path) in enumerate(zip(nodes, paths)):
        base = p.lens[b] - n
        for i, node in enumerate(path):
            sb, so = spot(p, b, base + node)
            db, do = spot(p, b, base + i)
            kc[db, :, do], vc[db, :, do] = p.kc[sb, :, so], p.vc[sb, :, so]
            if ks is not None:
                ks[db, :, :, do] = p.ks[sb, :, :, so]
    return kc, vc, ks


def accept(p, nodes, paths, width=None, new=True, stream=None):
    B = len(nodes)
    width = max([len(x) for x in paths] + [0]) if width is None else width
    path = torch.full((B, width), -9, dtype=torch.int32)
    for b, x in enumerate(paths):
        path[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
    starts = torch.tensor([3] + [3 + int(x) for x in torch.tensor(nodes).cumsum(0)],
                          dtype=torch.int32)
    lens = torch.tensor([len(x) for x in paths], dtype=torch.int32)
    out = torch.full((B,), -5, dtype=torch.int32, device="cuda") if new else None
    pkv.pkv_kv_accept_path(p.desc, p.kc, p.vc, p.tables, p.ctx, starts.cuda(), path.cuda(),
                           lens.cuda(), out, stream=stream)
    return out


def same(p, want):
    assert torch.equal(bytes_of(p.kc), bytes_of(want[0]))
    assert torch.equal(bytes_of(p.vc), bytes_of(want[1]))
    if want[2] is not None:
        assert torch.equal(bytes_of(p.ks), bytes_of(want[2]))


@pytest.mark.parametrize("cache,Hq,Hkv,d", [("f16", 4, 4, 64), ("bf16", 8, 2, 128),
                                            ("f16", 8, 1, 128), ("e4m3", 8, 4, 128),
                                            ("e4m3tok", 6, 3, 128)])
def test_paths(cache, Hq, Hkv, d):
    nodes = [1, 1, 7, 16, 33, 64, 64, 5, 0, 20]
    paths = [[], [0], [0, 2, 5], [15], list(range(33)), list(range(64)),
             [2 * i + 1 for i in range(32)], [4, 2, 0, 3, 1], [], [3, 3, 19, 0]]
    pasts = [5, 0, 9, 16, 1, 0, 100, 31, 0, 47]
    p = Paged([a + n for a, n in zip(pasts, nodes)], Hq, Hkv, d, cache, 5)
    want = expect(p, nodes, paths)
    new = accept(p, nodes, paths)
    same(p, want)
    assert new.tolist() == [a + len(x) for a, x in zip(pasts, paths)]
    assert p.err.item() == 0


def test_without_lengths_and_without_any_step():
    p = Paged([40, 50], 8, 2, 128, "bf16", 6)
    want = expect(p, [9, 9], [[1, 4], []])
    assert accept(p, [9, 9], [[1, 4], []], new=False) is None
    same(p, want)
    assert accept(p, [9, 9], [[], []], width=0).tolist() == [31, 41]
    same(p, want)


def test_what_breaks_the_rules_is_left_alone():
    nodes = [9, 9, 9, 9]
    p = Paged([40, 50, 60, 70], 8, 2, 128, "bf16", 7)
    p.ctx[1] = 8                      # shorter than its tree
    want = expect(p, nodes, [[5], [], [2, 1], [8, 0, 7]])
    path = [[5], [3], [2, 9, 1], [8, -1, 7]]
    # a node outside the tree: that step's row stays, the others move
    want = expect(p, nodes, [[5], [], [2, 1, 1], [8, 1, 7]])
    new = accept(p, nodes, path)
    same(p, want)
    assert new.tolist() == [32, -5, 54, 64]
    assert p.err.item() == pkv.PKV_ERR_BOUNDS


@pytest.mark.parametrize("bad", [-1, 10, 64])
def test_path_lengths_out_of_range(bad):
    p = Paged([40], 8, 2, 128, "bf16", 8)
    want = expect(p, [9], [[]])
    starts = torch.tensor([0, 9], dtype=torch.int32).cuda()
    path = torch.arange(20, dtype=torch.int32).flip(0).view(1, 20).contiguous().cuda()
    new = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    pkv.pkv_kv_accept_path(p.desc, p.kc, p.vc, p.tables, p.ctx, starts, path,
                           torch.tensor([bad], dtype=torch.int32).cuda(), new)
    same(p, want)
    assert new.item() == -5 and p.err.item() == pkv.PKV_ERR_BOUNDS


@pytest.mark.parametrize("first,last", [(9, 4), (-4, 5), (-9, 0), (2 ** 31 - 1, -2 ** 31),
                                        (2 ** 31 - 3, -2 ** 31 + 5)])
def test_starts_that_run_backwards_or_from_below_zero(first, last):
    """Also where the difference of the two, cut to 32 bits, is a count like another."""
    p = Paged([40], 8, 2, 128, "bf16", 12)
    want = expect(p, [9], [[]])
    new = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    pkv.pkv_kv_accept_path(p.desc, p.kc, p.vc, p.tables, p.ctx,
                           torch.tensor([first, last], dtype=torch.int32).cuda(),
                           torch.tensor([[0, 3]], dtype=torch.int32).cuda(),
                           torch.tensor([0], dtype=torch.int32).cuda(), new)
    same(p, want)
    assert new.item() == -5 and p.err.item() == pkv.PKV_ERR_BOUNDS


def test_blocks_outside_the_pool():
    p = Paged([60], 8, 2, 128, "bf16", 9)
    nodes, path = [40], [[30, 39, 25]]     # the tree lies at 20 .. 59
    want = expect(p, nodes, [[0, 1, 25]])  # the first two come from page 3
    p.tables[0, 3] = p.NB
    accept(p, nodes, path)
    same(p, want)
    assert p.err.item() == pkv.PKV_ERR_BOUNDS


def test_captured_and_replayed():
    p = Paged([45, 50], 8, 2, 128, "bf16", 10)
    starts = torch.tensor([0, 9, 20], dtype=torch.int32).cuda()
    path = torch.zeros(2, 6, dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pkv.pkv_kv_accept_path(p.desc, p.kc, p.vc, p.tables, p.ctx, starts, path, lens, new)
    for a, c in (([1, 3], [10, 9, 8, 0]), ([], [5]), ([8], [])):
        want = expect(p, [9, 11], [a, c])
        for b, x in enumerate((a, c)):
            path[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
            lens[b] = len(x)
        g.replay()
        torch.cuda.synchronize()
        same(p, want)
        assert new.tolist() == [36 + len(a), 39 + len(c)]
