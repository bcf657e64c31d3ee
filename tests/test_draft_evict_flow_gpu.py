"""The operators run together, as a serving loop makes the calls.

Drafting: a prompt, then rounds of a drafted tree per sequence (rotary append of its
nodes, tree attention, acceptance of a path), then a plain decode step over what was
kept.  Eviction: a prompt, then decode steps that add up weights, with an eviction
whenever the cache is full.

Every attention call is held to fp64 over the rows that the cache holds, read back
as stored and kept in lists by the rule of each operator; what the calls move is
compared exactly."""
import math

import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import CODE, DT, PAGE, half_step, rope_table

pytestmark = pytest.mark.gpu


class Server:
    def __init__(self, B, Hq, Hkv, d, cache, pages, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.__dict__.update(B=B, Hq=Hq, Hkv=Hkv, d=d, cache=cache, mbs=pages)
        NB = B * pages + 2
        self.NB = NB
        self.tables = torch.randperm(NB, generator=self.g)[:B * pages].view(B, pages).int()
        fp8 = cache.startswith("e4m3")
        self.dt = DT.get(cache, torch.bfloat16)
        self.kc = torch.full((NB, Hkv, PAGE, d), 0x7F if fp8 else float("nan"),
                             dtype=torch.uint8 if fp8 else self.dt, device="cuda")
        self.vc = self.kc.clone()
        self.ks = torch.full((NB, Hkv, 2, PAGE), float("nan"), device="cuda") \
            if cache == "e4m3tok" else None
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.desc = pkv.make_desc(NB, PAGE, Hkv, Hq, d, CODE[cache], self.ks, None, self.err)
        self.table = rope_table(4096, d).cuda()
        self.dtables = self.tables.cuda()
        self.scale = 1 / math.sqrt(d)

    def append(self, slots, positions):
        """New tokens with drawn q, k, v; their rotated q."""
        T = len(slots)
        qkv = torch.randn(T, self.Hq + 2 * self.Hkv, self.d, generator=self.g)
        q, k, v = qkv.to(self.dt).cuda().split([self.Hq, self.Hkv, self.Hkv], 1)
        out = torch.empty(T, self.Hq, self.d, dtype=self.dt, device="cuda")
        pkv.pkv_kv_append_rope(self.desc, self.kc, self.vc, torch.tensor(slots).cuda(),
                               torch.tensor(positions).cuda(), self.table, q, k, v, out)
        return out

    def slot(self, b, u):
        return int(self.tables[b, u // PAGE]) * PAGE + u % PAGE

    def row(self, b, u, h):
        """K and V of the row at index u under KV head h, fp64, as stored."""
        blk, off = int(self.tables[b, u // PAGE]), u % PAGE
        pair = []
        for i, c in enumerate((self.hk, self.hv)):
            x = c[blk, h, off]
            if self.ks is not None:
                x = x.view(torch.float8_e4m3fn).double() * self.hs[blk, h, i, off].double()
            pair.append(x.double())
        return pair

    def read_back(self):
        self.hk, self.hv = self.kc.cpu(), self.vc.cpu()
        self.hs = None if self.ks is None else self.ks.cpu()

    def attend(self, q, rows):
        """One query head over K, V rows (fp64): output, weights, and the errors that
        the calls may make (those of the operators' own tests)."""
        k, v = (torch.stack(x) for x in zip(*rows))
        s = k @ q * self.scale
        p = torch.softmax(s, 0)
        ds = (k.abs() @ q.abs() * self.scale).max() * self.d * 2.0 ** -23
        return p @ v, p, v.abs().max() * 2 * (ds + 2.0 ** -15), ds

    def close(self, got, ref, tol):
        bound = tol + half_step(ref.abs() + tol, "f32")
        assert ((got.double().cpu() - ref).abs() <= bound).all()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("cache,Hq,Hkv,d", [("bf16", 8, 2, 128), ("f16", 4, 4, 64)])
def test_drafted_trees_are_verified_and_accepted(cache, Hq, Hkv, d):
    s = Server(3, Hq, Hkv, d, cache, 16, 5)
    lens = [37, 1, 100]
    for b, n in enumerate(lens):
        s.append([s.slot(b, u) for u in range(n)], list(range(n)))
    ws = torch.full((pkv.pkv_tree_workspace_bytes(s.desc, 3, 64, s.mbs),), 0xff,
                    dtype=torch.uint8, device="cuda")
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    for step in range(4):
        nodes = [(7, 20, 1), (1, 64, 33), (16, 3, 40), (12, 5, 9)][step]
        words, slots, pos, parents = [], [], [], []
        for b, n in enumerate(nodes):
            up = [int(torch.randint(-1, j, (1,), generator=s.g)) if j else -1 for j in range(n)]
            depth, mine = [], []
            for j in range(n):
                depth.append(0 if up[j] < 0 else depth[up[j]] + 1)
                mine.append((mine[up[j]] if up[j] >= 0 else 0) | 1 << j)
            words += mine
            slots += [s.slot(b, lens[b] + j) for j in range(n)]
            pos += [lens[b] + x for x in depth]
            parents.append(up)
        q = s.append(slots, pos)
        ctx = i32([lens[b] + n for b, n in enumerate(nodes)])
        starts = i32([0] + torch.tensor(nodes).cumsum(0).tolist())
        mask = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words]).cuda()
        out = torch.empty(q.shape, device="cuda")
        pkv.pkv_paged_tree_attention(s.desc, q, s.kc, s.vc, s.dtables, ctx, starts, 64, mask,
                                     s.scale, out, ws)
        s.read_back()
        hq, r = q.double().cpu(), 0
        for b, n in enumerate(nodes):
            for j in range(n):
                see = list(range(lens[b])) + [lens[b] + i for i in range(n) if words[r] >> i & 1]
                for h in {0, Hq // 2, Hq - 1}:
                    kv = h // (Hq // Hkv)
                    ref, _, tol, _ = s.attend(hq[r, h], [s.row(b, u, kv) for u in see])
                    s.close(out[r, h], ref, tol)
                r += 1
        # a path from a root down to one of the nodes (in step 2 none for one sequence)
        paths = []
        for b, up in enumerate(parents):
            j = int(torch.randint(0, len(up), (1,), generator=s.g))
            path = []
            while j >= 0:
                path.insert(0, j)
                j = up[j]
            paths.append([] if step == 2 and b == 1 else path)
        width = max(len(x) for x in paths)
        path = torch.zeros(3, width, dtype=torch.int32)
        for b, x in enumerate(paths):
            path[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
        before = (s.hk, s.hv)
        pkv.pkv_kv_accept_path(s.desc, s.kc, s.vc, s.dtables, ctx, starts, path.cuda(),
                               i32([len(x) for x in paths]), new)
        s.read_back()
        for b, x in enumerate(paths):
            for i, node in enumerate(x):
                to, frm = (divmod(lens[b] + y, PAGE) for y in (i, node))
                for now, was in zip((s.hk, s.hv), before):
                    assert torch.equal(now[int(s.tables[b, to[0]]), :, to[1]],
                                       was[int(s.tables[b, frm[0]]), :, frm[1]])
            lens[b] += len(x)
        assert new.tolist() == lens
    # the next token of each sequence, over what was kept
    q = s.append([s.slot(b, lens[b]) for b in range(3)], lens)
    out = torch.empty(3, Hq, d, device="cuda")
    dws = torch.zeros(pkv.pkv_decode_workspace_bytes(s.desc, 3, s.mbs), dtype=torch.uint8,
                      device="cuda")
    pkv.pkv_paged_decode_attention(s.desc, q, s.kc, s.vc, s.dtables, new + 1, s.scale, out, dws)
    s.read_back()
    for b in range(3):
        for h in range(Hq):
            rows = [s.row(b, u, h // (Hq // Hkv)) for u in range(lens[b] + 1)]
            ref, _, tol, _ = s.attend(q[b, h].double().cpu(), rows)
            s.close(out[b, h], ref, tol)
    assert s.err.item() == 0


@pytest.mark.parametrize("cache,Hq,Hkv,d", [("bf16", 8, 2, 128), ("e4m3tok", 4, 2, 128)])
def test_decode_that_evicts_when_the_cache_is_full(cache, Hq, Hkv, d):
    budget, most, sinks, recent = 40, 48, 2, 10
    s = Server(2, Hq, Hkv, d, cache, most // PAGE, 7)
    lens, told = [45, 17], [45, 17]
    for b, n in enumerate(lens):
        s.append([s.slot(b, u) for u in range(n)], list(range(n)))
    i = dict(dtype=torch.int32, device="cuda")
    weights = torch.full((s.NB, Hkv, PAGE), float("nan"), device="cuda")
    positions = torch.full((s.NB, Hkv, PAGE), -1, **i)
    old, new = torch.zeros(2, **i), torch.zeros(2, **i)
    ws = torch.zeros(pkv.pkv_scored_workspace_bytes(s.desc, 2, s.mbs), dtype=torch.uint8,
                     device="cuda")
    # by sequence and KV head: the token of each row, and what it weighs (fp64), with
    # the error that the calls may have added up
    tokens = [[list(range(n)) for _ in range(Hkv)] for n in lens]
    heavy = [[torch.zeros(n, dtype=torch.float64) for _ in range(Hkv)] for n in lens]
    slack = [[torch.zeros(n, dtype=torch.float64) for _ in range(Hkv)] for n in lens]
    evictions = 0
    for step in range(30):
        q = s.append([s.slot(b, lens[b]) for b in range(2)], told)
        for b in range(2):
            for h in range(Hkv):
                tokens[b][h].append(told[b])
                heavy[b][h] = torch.cat([heavy[b][h], torch.zeros(1).double()])
                slack[b][h] = torch.cat([slack[b][h], torch.zeros(1).double()])
            lens[b] += 1
            told[b] += 1
        out = torch.empty(2, Hq, d, device="cuda")
        pkv.pkv_paged_decode_attention_scored(s.desc, q, s.kc, s.vc, s.dtables, i32(lens), weights,
                                              s.scale, out, ws, decay=1.0 if step else 0.0)
        s.read_back()
        hw = weights.double().cpu()
        for b in range(2):
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
        if max(lens) < most:
            continue
        evictions += 1
        pkv.pkv_kv_evict(s.desc, s.kc, s.vc, weights, positions, s.dtables, i32(lens), old,
                         i32(told), budget, sinks, recent, new)
        old = new.clone()
        before = (s.hk, s.hv, hw)
        s.read_back()
        hw = weights.double().cpu()
        hp = positions.cpu()
        for b in range(2):
            n = lens[b]
            keep = min(n, budget)
            for h in range(Hkv):
                at = torch.arange(n)
                blk, off = s.tables[b].long()[at // PAGE], at % PAGE
                w = before[2][blk, h, off]  # as the call saw them
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
    assert evictions >= 3 and s.err.item() == 0
