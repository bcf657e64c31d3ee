"""Eviction by accumulated weight: whole pools, byte for byte, against the rule
spelled out row by row."""
import numpy as np
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import PAGE, Paged

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lens, old, told, Hq=8, Hkv=2, d=128, cache="bf16", seed=1, weights="exp",
                 wider=0):
        self.p = p = Paged(lens, Hq, Hkv, d, cache, seed)
        if wider:  # a table with room for longer sequences
            p.tables = torch.cat([p.tables, torch.full((len(lens), wider), -3, dtype=torch.int32,
                                                       device="cuda")], 1).contiguous()
            p.mbs += wider
        g = torch.Generator().manual_seed(seed + 1000)
        shape = (p.NB, Hkv, PAGE)
        if weights == "exp":
            w = torch.exp(2 * torch.randn(shape, generator=g))
        elif weights == "few":  # many ties
            w = torch.randint(0, 4, shape, generator=g).float()
        elif weights == "same":
            w = torch.full(shape, 0.25)
        else:  # everything a float can be
            pick = torch.tensor([0.0, -0.0, 1e-42, -1e-42, 1.0, -1.0, float("inf"),
                                 -float("inf"), float("nan"), 3e38, 2.0 ** -126])
            w = pick[torch.randint(0, len(pick), shape, generator=g)]
        self.w = w.cuda()
        self.pos = torch.randint(0, 1 << 30, shape, generator=g, dtype=torch.int32).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.old, self.told = torch.tensor(old, **i32), torch.tensor(told, **i32)
        for b, (n, o, t) in enumerate(zip(lens, old, told)):
            for h in range(Hkv):  # distinct positions before those of the new rows
                some = torch.randperm(max(1, t - (n - o)), generator=g)[:o].to(torch.int32)
                u = torch.arange(o)
                self.pos[p.tables[b].cpu().long()[u // PAGE], h, u % PAGE] = some.cuda()
        self.new = torch.full((len(lens),), -5, **i32)

    def run(self, budget, sinks, recent, stream=None):
        p = self.p
        pkv.pkv_kv_evict(p.desc, p.kc, p.vc, self.w, self.pos, p.tables, p.ctx, self.old,
                         self.told, budget, sinks, recent, self.new, stream=stream)

    def pools(self):
        p = self.p
        return [bytes_of(t).clone() for t in (p.kc, p.vc, self.w, self.pos)] + \
            ([bytes_of(p.ks).clone()] if p.cache == "e4m3tok" else [])

    def expect(self, budget, sinks, recent, bad=(), skip=()):
        """The pools after the call.  bad: (sequence, page) outside the pool; skip:
        sequences whose lengths break the rules."""
        p = self.p
        kc, vc = (x.clone().view(torch.uint8).reshape(p.NB, p.Hkv, PAGE, -1)
                  for x in (p.kc, p.vc))
        w, pos = self.w.clone(), self.pos.clone()
        ks = p.ks.clone() if p.cache == "e4m3tok" else None
        new = self.new.tolist()
        for b, n in enumerate(p.lens):
            if b in skip:
                continue
            new[b] = min(n, budget)
            o, t = int(self.old[b]), int(self.told[b])
            u = np.arange(n)
            table = p.tables[b].cpu().long()
            ok = np.array([(b, i // PAGE) not in bad for i in u], dtype=bool)
            blk, off = table[torch.from_numpy(u // PAGE)], torch.from_numpy(u % PAGE)
            blk = torch.where(torch.from_numpy(ok), blk, 0)
            for h in range(p.Hkv):
                at = self.pos[blk, h, off].cpu().numpy()
                at = np.where(u >= o, t - n + u, at)
                late = torch.from_numpy((u >= o) & ok)
                pos[blk[late], h, off[late]] = torch.from_numpy(at.astype(np.int32))[late].cuda()
                if n <= budget:
                    continue
                wt = self.w[blk, h, off].cpu().numpy().astype(np.float64)
                # NaN above infinity, guarded above all, outside the pool below all
                rank = np.zeros(n)
                rank[np.isnan(wt)] = 1
                rank[(at < sinks) | (at >= t - recent)] = 2
                rank[~ok] = -1
                wt = np.where(rank == 0, wt, 0.0)
                best = np.lexsort((u, -wt, -rank))[:budget]
                keep = np.zeros(n, dtype=bool)
                keep[best] = True
                holes, movers = u[~keep & (u < budget)], u[keep & (u >= budget)]
                assert len(holes) == len(movers)
                go = ok[holes] & ok[movers]
                holes, movers = holes[go], movers[go]
                db, do, sb, so = blk[holes], off[holes], blk[movers], off[movers]
                kc[db, h, do], vc[db, h, do] = kc[sb, h, so], vc[sb, h, so]
                w[db, h, do] = w[sb, h, so]
                pos[db, h, do] = torch.from_numpy(at[movers].astype(np.int32)).cuda()
                if ks is not None:
                    ks[db, h, :, do] = ks[sb, h, :, so]
        return [bytes_of(x) for x in (kc, vc, w, pos)] + \
            ([] if ks is None else [bytes_of(ks)]), new

    def check(self, budget, sinks, recent, bad=(), skip=()):
        want, new = self.expect(budget, sinks, recent, bad, skip)
        self.run(budget, sinks, recent)
        for name, a, b in zip(("k", "v", "weights", "positions", "scales"), self.pools(), want):
            assert torch.equal(a.reshape(-1), b.reshape(-1)), name
        assert self.new.tolist() == new


def bytes_of(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("cache,Hq,Hkv,d", [("f16", 4, 4, 64), ("bf16", 8, 2, 128),
                                            ("e4m3", 8, 1, 128), ("e4m3tok", 6, 3, 128)])
@pytest.mark.parametrize("weights", ["exp", "few"])
def test_prompts(cache, Hq, Hkv, d, weights):
    lens = [1, 0, 99, 100, 101, 117, 128, 500, 33, 1000]
    c = Case(lens, [0] * 10, lens, Hq, Hkv, d, cache, 3, weights)
    c.check(100, 4, 20)
    assert c.p.err.item() == 0


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 0, 64),
                                                 (64, 64, 0), (64, 30, 34), (63, 5, 10),
                                                 (2000, 4, 500)])
def test_budgets(budget, sinks, recent):
    lens = [257, 64, 65, 63, 3000]
    c = Case(lens, [0, 10, 64, 63, 1500], [257, 400, 65, 63, 9000], seed=5)
    c.check(budget, sinks, recent)


@pytest.mark.parametrize("weights", ["same", "all", "few"])
def test_ties_and_every_kind_of_float(weights):
    lens = [700, 2049, 130]
    c = Case(lens, [0, 1000, 130], [700, 5000, 400], seed=7, weights=weights)
    c.check(100, 3, 9)


def test_again_and_again():
    """A cache that is full: some rows come at every step, as many go."""
    budget, fresh = 200, 7
    lens = [budget + fresh] * 3
    c = Case(lens, [0] * 3, lens, Hkv=2, seed=9)
    g = torch.Generator().manual_seed(10)
    for step in range(6):
        c.check(budget, 4, 50)
        c.old = c.new.clone()
        c.told = c.told + fresh
        for b in range(3):  # the rows behind the budget are new ones
            for u in range(budget, budget + fresh):
                blk, off = int(c.p.tables[b, u // PAGE]), u % PAGE
                c.p.kc[blk, :, off] = torch.randn(2, 128, generator=g).bfloat16().cuda()
                c.p.vc[blk, :, off] = torch.randn(2, 128, generator=g).bfloat16().cuda()
                c.w[blk, :, off] = torch.rand(2, generator=g).cuda()
    # the sinks are all there
    for b in range(3):
        u = torch.arange(budget)
        for h in range(2):
            have = c.pos[c.p.tables[b].cpu().long()[u // PAGE], h, u % PAGE].cpu()
            assert set(range(4)) <= set(have.tolist()) and len(set(have.tolist())) == budget
            assert set(range(int(c.told[b]) - fresh - 50, int(c.told[b]) - fresh)) <= \
                set(have.tolist())


@pytest.mark.parametrize("Hkv,n,budget,weights", [(1, 70001, 5000, "exp"), (1, 70001, 60000, "few"),
                                                  (3, 20000, 10000, "same"), (2, 5000, 17, "all"),
                                                  (8, 40000, 1, "exp")])
def test_long_sequences_over_several_ctas(Hkv, n, budget, weights):
    c = Case([n], [0], [n], Hq=Hkv, Hkv=Hkv, d=64, cache="f16", seed=11, weights=weights)
    c.check(budget, min(4, budget - 1), budget // 8)


def test_a_table_far_wider_than_the_sequences():
    c = Case([300, 90], [0, 0], [300, 90], seed=13, wider=9000)
    c.check(128, 4, 16)


def test_batches_larger_than_the_gpu():
    g = torch.Generator().manual_seed(14)
    lens = torch.randint(0, 200, (300,), generator=g).tolist()
    c = Case(lens, [0] * 300, lens, Hq=4, Hkv=2, d=64, cache="f16", seed=15)
    c.check(64, 2, 10)


def test_blocks_outside_the_pool():
    lens = [300, 200, 16]
    c = Case(lens, [0, 100, 0], [300, 900, 16], seed=17)
    bad = [(0, 2), (0, 18), (1, 12), (2, 0)]
    for i, (b, page) in enumerate(bad):
        c.p.tables[b, page] = (-1, c.p.NB, 1 << 30, -(1 << 31))[i]
    c.check(100, 4, 20, bad=set(bad))
    assert c.p.err.item() == pkv.PKV_ERR_BOUNDS


def test_a_budget_that_has_to_keep_rows_outside_the_pool():
    c = Case([64], [0], [64], seed=18)
    bad = {(0, 0), (0, 1), (0, 3)}
    for b, page in bad:
        c.p.tables[b, page] = -1
    c.check(40, 4, 10, bad=bad)


def test_lengths_that_break_the_rules():
    lens = [300] * 5
    c = Case(lens, [0] * 5, lens, seed=19)
    c.p.ctx[0], c.p.ctx[1] = -1, c.p.mbs * PAGE + 1
    c.old[2] = 301
    c.told[3] = 299
    c.check(100, 4, 20, skip={0, 1, 2, 3})
    assert c.p.err.item() == pkv.PKV_ERR_BOUNDS


def test_captured_and_replayed_with_other_lengths():
    c = Case([400, 300], [0, 0], [400, 300], seed=21)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.run(120, 4, 30)
    for lens, told in (([400, 300], [400, 300]), ([121, 119], [500, 119]), ([120, 260], [800, 900])):
        c.p.lens = lens
        c.p.ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        c.told.copy_(torch.tensor(told, dtype=torch.int32))
        want, new = c.expect(120, 4, 30)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(c.pools(), want):
            assert torch.equal(a.reshape(-1), b.reshape(-1))
        assert c.new.tolist() == new


@pytest.mark.parametrize("wider", [20000, 49133])
def test_the_widest_tables(wider):
    """Clusters of eight and of sixteen, most of whose CTAs have no row."""
    c = Case([300, 90], [0, 0], [300, 90], seed=23, wider=wider)
    c.check(128, 4, 16)


def test_two_streams():
    """Calls on pools of their own, queued side by side."""
    cases = [Case([900 + 31 * i] * 6, [0] * 6, [900 + 31 * i] * 6, seed=25 + i) for i in range(2)]
    wants = [c.expect(500, 4, 100) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c, st in zip(cases, streams):
        c.run(500, 4, 100, stream=st)
    torch.cuda.synchronize()
    for c, (want, new) in zip(cases, wants):
        for a, b in zip(c.pools(), want):
            assert torch.equal(a.reshape(-1), b.reshape(-1))
        assert c.new.tolist() == new
