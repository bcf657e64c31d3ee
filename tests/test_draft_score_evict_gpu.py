"""Drafting and eviction in one loop: a tree of drafts is verified and a path of it
accepted, the accepted rows' weights are set to zero, a scored step follows, and the
cache is cut down when it is full.  Slots that hold no row weigh NaN at every step, as
slots of a pool that others used before may."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import PAGE
from test_draft_evict_flow_gpu import Server, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,Hq,Hkv,d", [("bf16", 8, 2, 128), ("f16", 4, 4, 64)])
def test_accepted_rows_take_part_in_the_eviction(cache, Hq, Hkv, d):
    budget, full, sinks, recent, B = 40, 46, 2, 10, 2
    s = Server(B, Hq, Hkv, d, cache, 5, 9)
    lens, told = [30, 39], [30, 39]
    for b, n in enumerate(lens):
        s.append([s.slot(b, u) for u in range(n)], list(range(n)))
    i = dict(dtype=torch.int32, device="cuda")
    weights = torch.full((s.NB, Hkv, PAGE), float("nan"), device="cuda")
    positions = torch.full((s.NB, Hkv, PAGE), -1, **i)
    old, new = torch.zeros(B, **i), torch.zeros(B, **i)
    tws = torch.zeros(pkv.pkv_tree_workspace_bytes(s.desc, B, 8, s.mbs), dtype=torch.uint8,
                      device="cuda")
    sws = torch.zeros(pkv.pkv_scored_workspace_bytes(s.desc, B, s.mbs), dtype=torch.uint8,
                      device="cuda")
    tokens = [[list(range(n)) for _ in range(Hkv)] for n in lens]
    heavy = [[torch.zeros(n, dtype=torch.float64) for _ in range(Hkv)] for n in lens]
    slack = [[torch.zeros(n, dtype=torch.float64) for _ in range(Hkv)] for n in lens]
    path = i32([[1, 3, 6], [0, 2, 7]])          # of eight nodes each
    evictions = 0

    def came(b, count):  # the next `count` tokens have rows from now on
        for h in range(Hkv):
            tokens[b][h] += range(told[b], told[b] + count)
            heavy[b][h] = torch.cat([heavy[b][h], torch.zeros(count).double()])
            slack[b][h] = torch.cat([slack[b][h], torch.zeros(count).double()])
        lens[b] += count
        told[b] += count

    for step in range(12):
        # ---- eight drafts behind each sequence, one of their paths kept
        q = s.append([s.slot(b, lens[b] + j) for b in range(B) for j in range(8)],
                     [told[b] + j for b in range(B) for j in range(8)])
        ctx, starts = i32([n + 8 for n in lens]), i32([0, 8, 16])
        mask = torch.tensor([(2 << j) - 1 for j in range(8)] * B).cuda()
        out = torch.empty(q.shape, device="cuda")
        pkv.pkv_paged_tree_attention(s.desc, q, s.kc, s.vc, s.dtables, ctx, starts, 8, mask,
                                     s.scale, out, tws)
        took = [1 + (step + b) % 3 for b in range(B)]
        pkv.pkv_kv_accept_path(s.desc, s.kc, s.vc, s.dtables, ctx, starts, path, i32(took), new)
        for b in range(B):
            for u in range(lens[b], lens[b] + took[b]):  # the caller's part
                weights[int(s.tables[b, u // PAGE]), :, u % PAGE] = 0.0
            came(b, took[b])
        assert new.tolist() == lens
        # ---- the next token
        q = s.append([s.slot(b, lens[b]) for b in range(B)], told)
        for b in range(B):
            came(b, 1)
        out = torch.empty(B, Hq, d, device="cuda")
        pkv.pkv_paged_decode_attention_scored(s.desc, q, s.kc, s.vc, s.dtables, i32(lens), weights,
                                              s.scale, out, sws, decay=1.0 if step else 0.0)
        s.read_back()
        hw = weights.double().cpu()
        for b in range(B):
            n = lens[b]
            at = torch.arange(n)
            blk = s.tables[b].long()[at // PAGE]
            for h in range(Hkv):
                rows = [s.row(b, u, h) for u in range(n)]
                for x in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                    ref, p, tol, ds = s.attend(q[b, x].double().cpu(), rows)
                    s.close(out[b, x], ref, tol)
                    heavy[b][h] += p
                    slack[b][h] += p * (2 * ds + 2.0 ** -20 + n * 2.0 ** -24)
                slack[b][h] += 2.0 ** -23 * heavy[b][h] + 1e-37
                assert ((hw[blk, h, at % PAGE] - heavy[b][h]).abs() <= slack[b][h]).all()
        if max(lens) >= full:
            evictions += 1
            before = (s.hk, s.hv, hw)
            pkv.pkv_kv_evict(s.desc, s.kc, s.vc, weights, positions, s.dtables, i32(lens), old,
                             i32(told), budget, sinks, recent, new)
            old = new.clone()
            s.read_back()
            hw, hp = weights.double().cpu(), positions.cpu()
            for b in range(B):
                n, keep = lens[b], min(lens[b], budget)
                for h in range(Hkv):
                    at = torch.arange(n)
                    blk, off = s.tables[b].long()[at // PAGE], at % PAGE
                    w = before[2][blk, h, off]
                    rank = [(0 if t < sinks or t >= told[b] - recent else 1, -float(w[u]), u)
                            for u, t in enumerate(tokens[b][h])]
                    kept = sorted(x[2] for x in sorted(rank)[:keep])
                    holes = [u for u in range(keep) if u not in kept]
                    src = list(range(keep))
                    for hole, u in zip(holes, [u for u in kept if u >= keep]):
                        src[hole] = u
                    t = torch.tensor(src)
                    for now, was in zip((s.hk, s.hv), before):
                        assert torch.equal(now[blk[:keep], h, off[:keep]], was[blk[t], h, off[t]])
                    assert torch.equal(hw[blk[:keep], h, off[:keep]], w[t])
                    tokens[b][h] = [tokens[b][h][u] for u in src]
                    heavy[b][h], slack[b][h] = heavy[b][h][t], slack[b][h][t]
                    assert hp[blk[:keep], h, off[:keep]].tolist() == tokens[b][h]
                lens[b] = keep
            assert new.tolist() == lens
        for b in range(B):  # whoever had these slots before
            for u in range(lens[b], s.mbs * PAGE):
                weights[int(s.tables[b, u // PAGE]), :, u % PAGE] = float("nan")
    assert evictions >= 3 and s.err.item() == 0
