"""pkv_kv_append_rope against the rotation formula in 64 bits, and against
pkv_kv_append where the rotation is the identity."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import CODE, DT, PAGE, half_step, rope_table, rotate

pytestmark = pytest.mark.gpu


class Append:
    def __init__(self, T, Hq, Hkv, d, rot, cache, seed, interleaved=False, fused=True, max_pos=500):
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(T=T, Hq=Hq, Hkv=Hkv, d=d, rot=rot, cache=cache,
                             interleaved=interleaved)
        self.dt = DT.get(cache, torch.bfloat16)
        NB = (2 * T + PAGE - 1) // PAGE + 2
        self.NB = NB
        fp8 = cache.startswith("e4m3")
        fill = torch.randint(0, 120, (NB, Hkv, PAGE, d), generator=g, dtype=torch.uint8)
        self.k0 = fill if fp8 else torch.randn(fill.shape, generator=g).to(DT[cache])
        self.v0 = self.k0.flip(0).contiguous()
        self.s0 = {"e4m3": torch.rand(Hkv, generator=g) / 50 + 0.005,
                   "e4m3tok": torch.rand(NB, Hkv, 2, PAGE, generator=g)}.get(cache)
        vs = torch.rand(Hkv, generator=g) / 50 + 0.005 if cache == "e4m3" else None
        qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(self.dt)
        self.slots = torch.randperm(NB * PAGE, generator=g)[:T]
        self.pos = torch.randint(0, max_pos, (T,), generator=g)
        self.table = rope_table(max_pos, rot)
        self.qh, self.kh, self.vh = (x.double() for x in
                                     qkv.split([Hq, Hkv, Hkv], dim=1))
        dev = qkv.cuda()
        parts = dev.split([Hq, Hkv, Hkv], dim=1)
        self.q, self.k, self.v = parts if fused else [x.contiguous() for x in parts]
        self.kc, self.vc = self.k0.cuda(), self.v0.cuda()
        self.ks = None if self.s0 is None else self.s0.cuda()
        self.vs = None if vs is None else vs.cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.desc = pkv.make_desc(NB, PAGE, Hkv, Hq, d, CODE[cache], self.ks, self.vs, self.err)
        self.q_out = torch.full((T, Hq, d), 7.0, dtype=self.dt, device="cuda")
        self.dslots, self.dpos, self.dtable = self.slots.cuda(), self.pos.cuda(), self.table.cuda()

    def run(self, **kw):
        pkv.pkv_kv_append_rope(self.desc, self.kc, self.vc, self.dslots, self.dpos, self.dtable,
                               self.q, self.k, self.v, kw.pop("q_out", self.q_out),
                               interleaved=self.interleaved, **kw)

    def check(self, rows=None, q_rows=None, q_out=None):
        """rows: tokens whose k and v were written (all); the rest of the
        cache is as it was."""
        rows = range(self.T) if rows is None else rows
        q_rows = list(range(self.T) if q_rows is None else q_rows)
        # two products and a sum in fp32: 2^-23 of |x0| + |x1|, then half a step
        name = {torch.float16: "f16", torch.bfloat16: "bf16"}[self.dt]
        ok_pos = self.pos.clamp(0, len(self.table) - 1)
        yq = rotate(self.qh, self.table, ok_pos, self.interleaved)
        got = (self.q_out if q_out is None else q_out).double().cpu()
        arith = 2.0 ** -22 * self.qh.abs().amax(-1, keepdim=True)
        off = (got - yq).abs() - half_step(yq.abs() + arith, name) - arith
        if q_rows:
            assert off[q_rows].max() <= 0
        left = [t for t in range(self.T) if t not in set(q_rows)]
        assert torch.all(got[left] == 7.0)
        yk = rotate(self.kh, self.table, ok_pos, self.interleaved)
        for i, (cache, before, y, src) in enumerate(((self.kc, self.k0, yk, self.kh),
                                                     (self.vc, self.v0, self.vh, self.vh))):
            want = before.clone()
            now = cache.cpu()
            for t in rows:
                blk, off = int(self.slots[t]) // PAGE, int(self.slots[t]) % PAGE
                row = now[blk, :, off]
                arith = 2.0 ** -22 * src[t].abs().amax(-1, keepdim=True)
                if not self.cache.startswith("e4m3"):
                    bound = half_step(y[t].abs() + arith, name) + (arith if i == 0 else 0)
                    assert ((row.double() - y[t]).abs() <= bound).all()
                else:
                    if self.cache == "e4m3":
                        s = (self.ks if i == 0 else self.vs).cpu().double()[:, None]
                    else:
                        s = self.ks.cpu()[blk, :, i, off].double()[:, None]
                        top = y[t].abs().amax(-1, keepdim=True) / 448
                        assert ((s - top).abs() <= top * 2.0 ** -23 + arith / 448).all()
                    z = (y[t] / s).clamp(-448, 448)
                    code = row.view(torch.float8_e4m3fn).double()
                    slack = arith / s + z.abs() * 2.0 ** -23
                    # the slack may also carry a value over the next border
                    assert ((code - z).abs() <= half_step(z.abs() + slack, "e4m3") + slack).all()
                want[blk, :, off] = row
            same = want.view(torch.uint8) == now.view(torch.uint8)
            assert same.all()  # nothing else was touched


CASES = [  # T, Hq, Hkv, d, rot, cache, interleaved, fused projection
    (1, 32, 8, 128, 128, "bf16", False, True),
    (3, 8, 8, 64, 64, "f16", False, False),
    (37, 6, 3, 64, 32, "f16", True, True),
    (70, 16, 2, 128, 96, "bf16", False, True),
    (70, 16, 2, 128, 16, "bf16", True, True),
    (129, 4, 4, 128, 128, "e4m3", False, True),
    (45, 8, 1, 128, 64, "e4m3", True, False),
    (33, 8, 2, 128, 128, "e4m3tok", False, True),
    (18, 24, 3, 128, 32, "e4m3tok", True, True),
    (700, 32, 8, 128, 128, "bf16", False, True),
]


@pytest.mark.parametrize("case", CASES)
def test_matches_the_formula(case):
    T, Hq, Hkv, d, rot, cache, inter, fused = case
    a = Append(T, Hq, Hkv, d, rot, cache, 5 + T, inter, fused)
    a.run()
    torch.cuda.synchronize()
    assert a.err.item() == 0
    a.check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e4m3tok"])
def test_padding_and_bad_tokens(cache):
    """A negative slot keeps the token's k and v out of the cache, a slot past
    the pool does so and is reported, a position outside the table writes
    nothing at all and is reported."""
    a = Append(40, 8, 2, 128, 128, cache, 9)
    slots, pos = a.slots.clone(), a.pos.clone()
    slots[3] = -1
    slots[39] = -(2 ** 40)
    a.slots, a.dslots = slots, slots.cuda()
    a.run()
    assert a.err.item() == 0
    good = [t for t in range(40) if t not in (3, 39)]
    a.check(rows=good)
    b = Append(40, 8, 2, 128, 128, cache, 9)
    slots = b.slots.clone()
    slots[5] = b.NB * PAGE
    slots[6] = 2 ** 45
    pos = b.pos.clone()
    pos[7], pos[8], pos[0] = -1, 500, 2 ** 50
    b.slots, b.dslots, b.pos, b.dpos = slots, slots.cuda(), pos, pos.cuda()
    b.run()
    assert b.err.item() == pkv.PKV_ERR_BOUNDS
    b.check(rows=[t for t in range(40) if t not in (0, 5, 6, 7, 8)],
            q_rows=[t for t in range(40) if t not in (0, 7, 8)])


@pytest.mark.parametrize("cache,d", [("f16", 64), ("bf16", 128), ("e4m3", 128),
                                     ("e4m3tok", 128)])
def test_without_rotation_it_is_the_append(cache, d):
    """Cosines of one and sines of zero: every byte that pkv_kv_append writes
    (all-zero rows among them), and q unchanged."""
    a = Append(77, 8, 2, d, d, cache, 21, fused=False)
    a.k[4], a.v[5] = 0, 0
    a.dtable[:, :d // 2], a.dtable[:, d // 2:] = 1.0, 0.0
    a.run()
    b = Append(77, 8, 2, d, d, cache, 21, fused=False)
    b.k[4], b.v[5] = 0, 0
    pkv.pkv_kv_append(b.desc, b.kc, b.vc, b.dslots, b.k, b.v)
    assert torch.equal(a.kc.view(torch.uint8), b.kc.view(torch.uint8))
    assert torch.equal(a.vc.view(torch.uint8), b.vc.view(torch.uint8))
    if cache == "e4m3tok":
        assert torch.equal(a.ks, b.ks)
    assert torch.equal(a.q_out, a.q)


def test_in_place_and_empty():
    a = Append(50, 8, 2, 128, 64, "bf16", 31, fused=False)
    a.run(q_out=a.q)
    a.check(q_out=a.q)
    n = Append(1, 8, 2, 128, 64, "bf16", 32)
    pkv.pkv_kv_append_rope(n.desc, n.kc, n.vc, n.dslots[:0], n.dpos[:0], n.dtable, n.q[:0],
                           n.k[:0], n.v[:0], n.q_out[:0])
    assert torch.equal(n.kc.cpu(), n.k0)


def test_captured_on_another_stream():
    """Captured once on a side stream, replayed on new inputs."""
    a = Append(64, 8, 2, 128, 128, "e4m3tok", 41)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        a.run()
    other = Append(64, 8, 2, 128, 128, "e4m3tok", 42)
    for name in ("q", "k", "v"):
        getattr(a, name).copy_(getattr(other, name))
    a.dpos.copy_(other.dpos)
    a.dslots.copy_(other.dslots)
    graph.replay()
    torch.cuda.synchronize()
    a.qh, a.kh, a.vh, a.pos, a.slots = other.qh, other.kh, other.vh, other.pos, other.slots
    a.check()


def test_slots_past_32_bits_of_bytes():
    """A pool whose later rows lie past 2^32 bytes."""
    NB, Hkv, d = 40000, 32, 128  # 40000 x 32 x 16 x 128 bf16: 5.2 GB a cache
    kc = torch.zeros(NB, Hkv, PAGE, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    desc = pkv.make_desc(NB, PAGE, Hkv, Hkv, d, pkv.PKV_BF16)
    q, k, v = (torch.randn(2, Hkv, d, device="cuda").bfloat16() for _ in range(3))
    slots = torch.tensor([NB * PAGE - 1, 38000 * PAGE], device="cuda")
    pos = torch.tensor([3, 499], device="cuda")
    table = rope_table(500, d)
    out = torch.empty_like(q)
    pkv.pkv_kv_append_rope(desc, kc, vc, slots, pos, table.cuda(), q, k, v, out)
    y = rotate(k.double().cpu(), table, pos.cpu(), False)
    for t, (blk, off) in enumerate(((NB - 1, 15), (38000, 0))):
        got = kc[blk, :, off].double().cpu()
        bound = half_step(y[t], "bf16") + 2.0 ** -22 * k[t].double().cpu().abs().amax()
        assert ((got - y[t]).abs() <= 1.01 * bound).all()
        assert torch.equal(vc[blk, :, off], v[t])
    assert kc.count_nonzero().item() <= 2 * Hkv * d
