"""The cache's tree, acceptance, scored and eviction calls on blocks whose bytes lie
past 4 GB from the start of the pool (element offsets past 2^31)."""
import math

import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import PAGE, Paged, check
from test_scored_decode_gpu import check_weights
from test_scored_decode_gpu import expect as expect_scored
from test_tree_attention_gpu import as_int64, expect, starts_of, trees

pytestmark = pytest.mark.gpu

NB, HKV, D = 140_000, 8, 128   # 4.6 GB per cache


@pytest.fixture(scope="module")
def large():
    """A small pool's sequences moved to the last blocks of a large one."""
    p = Paged([300, 70, 129], 16, HKV, D, "bf16", 5)
    kc = torch.empty(NB, HKV, PAGE, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    assert (NB - p.NB) * HKV * PAGE * D > 1 << 31
    kc[NB - p.NB:], vc[NB - p.NB:] = p.kc, p.vc
    p.tables = torch.where(p.tables >= 0, p.tables + (NB - p.NB), p.tables).int().contiguous()
    p.kc, p.vc, p.NB = kc, vc, NB
    p.desc = pkv.make_desc(NB, PAGE, HKV, 16, D, pkv.PKV_BF16, err_word=p.err)
    p.scale = 1 / math.sqrt(D)
    return p


def test_tree(large):
    p, nodes = large, [40, 3, 64]
    words = trees(nodes, 6)
    q = p.queries(sum(nodes), 7, 2.0)
    out = torch.empty(q.shape, device="cuda")
    ws = torch.zeros(pkv.pkv_tree_workspace_bytes(p.desc, 3, 64, p.mbs), dtype=torch.uint8,
                     device="cuda")
    pkv.pkv_paged_tree_attention(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx,
                                 starts_of(nodes).cuda(), 64, as_int64(words).cuda(), p.scale,
                                 out, ws)
    check(out, *expect(p, q, nodes, words), "f32")


def test_scored(large):
    p = large
    weights = torch.zeros(NB, HKV, PAGE, device="cuda")
    q = p.queries(3, 8, 2.0)
    ref, tol, w, wt = expect_scored(p, q, weights, 1.0)
    out = torch.empty(q.shape, device="cuda")
    ws = torch.zeros(pkv.pkv_scored_workspace_bytes(p.desc, 3, p.mbs), dtype=torch.uint8,
                     device="cuda")
    pkv.pkv_paged_decode_attention_scored(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, weights,
                                          p.scale, out, ws)
    check(out, ref, tol, "f32")
    check_weights(weights, w, wt)


def test_accept_then_evict(large):
    p, tables = large, large.tables.cpu().long()
    rows = [(p.kc[tables[b, :-(-n // PAGE)]].transpose(1, 2).reshape(-1, HKV, D)[:n].clone(),
             p.vc[tables[b, :-(-n // PAGE)]].transpose(1, 2).reshape(-1, HKV, D)[:n].clone())
            for b, n in enumerate(p.lens)]
    nodes, paths = [20, 9, 64], [[3, 19], [8], [0, 63, 5]]
    path = torch.zeros(3, 3, dtype=torch.int32)
    for b, x in enumerate(paths):
        path[b, :len(x)] = torch.tensor(x)
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    pkv.pkv_kv_accept_path(p.desc, p.kc, p.vc, p.tables, p.ctx, starts_of(nodes).cuda(),
                           path.cuda(), torch.tensor([2, 1, 3], dtype=torch.int32).cuda(), new)
    src = [list(range(n - k)) + [n - k + i for i in x]
           for n, k, x in zip(p.lens, nodes, paths)]
    assert new.tolist() == [len(x) for x in src]
    # then an eviction that keeps the last 30 rows and the 20 first of the others
    lens = new.clone()
    weights = torch.zeros(NB, HKV, PAGE, device="cuda")
    positions = torch.zeros(NB, HKV, PAGE, dtype=torch.int32, device="cuda")
    pkv.pkv_kv_evict(p.desc, p.kc, p.vc, weights, positions, p.tables, lens,
                     torch.zeros_like(lens), lens, 50, 0, 30, new)
    assert new.tolist() == [50, 50, 50] and p.err.item() == 0
    for b, x in enumerate(src):
        n = len(x)
        kept = list(range(20)) + list(range(n - 30, n))
        holes = [u for u in range(50) if u not in kept]
        at = list(range(50))
        for hole, u in zip(holes, [u for u in kept if u >= 50]):
            at[hole] = u
        blk, off = tables[b][torch.arange(50) // PAGE], torch.arange(50) % PAGE
        want = torch.tensor([x[u] for u in at])
        for cache, row in zip((p.kc, p.vc), rows[b]):
            assert torch.equal(cache[blk, :, off], row[want])
        assert positions[blk, 0, off].tolist() == at
