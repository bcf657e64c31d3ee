"""The rotary append with the attention calls that read what it wrote, as a
serving loop makes them: prompts in chunks, then token by token.

The reference rotates, in fp64, the same drawn q, k and v and attends in fp64.
Its keys and queries are rounded to the cache's type as the calls round theirs;
where fp32 and fp64 land on two sides of a rounding border, one element of a row
is a step off, which moves a score by at most 2^-7 |q_i k_i| scale: the bound
below grants every score one such element of q and one of k."""
import math

import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import CODE, DT, PAGE, attend, half_step, rope_table, rotate

pytestmark = pytest.mark.gpu


class Server:
    """B sequences over one pool; tables hold whole pages, dealt out as needed."""

    def __init__(self, B, Hq, Hkv, d, rot, cache, pages, prefix_pages=0, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.__dict__.update(B=B, Hq=Hq, Hkv=Hkv, d=d, rot=rot, dt=DT[cache], cache=cache)
        NB = prefix_pages + B * pages + 2
        perm = torch.randperm(NB, generator=self.g).to(torch.int32)
        self.prefix = perm[:prefix_pages]
        own = perm[prefix_pages:prefix_pages + B * pages].view(B, pages)
        self.tables = torch.cat([self.prefix[None].expand(B, -1), own], 1).contiguous()
        self.kc = torch.full((NB, Hkv, PAGE, d), float("nan"), dtype=self.dt, device="cuda")
        self.vc = self.kc.clone()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.desc = pkv.make_desc(NB, PAGE, Hkv, Hq, d, CODE[cache], err_word=self.err)
        self.table = rope_table(8192, rot)
        self.dtable, self.dtables = self.table.cuda(), self.tables.cuda()
        self.scale = 1 / math.sqrt(d)
        self.K = [torch.zeros(0, Hkv, d, dtype=torch.float64) for _ in range(B)]
        self.V = [x.clone() for x in self.K]

    def new(self, T, gain):
        qkv = torch.randn(T, self.Hq + 2 * self.Hkv, self.d, generator=self.g)
        qkv[:, :self.Hq] *= gain
        return qkv.to(self.dt)

    def slots(self, b, pos):
        return self.tables[b, pos // PAGE].long() * PAGE + pos % PAGE

    def append(self, qkv, slots, pos):
        q, k, v = qkv.cuda().split([self.Hq, self.Hkv, self.Hkv], 1)
        out = torch.empty(len(pos), self.Hq, self.d, dtype=self.dt, device="cuda")
        pkv.pkv_kv_append_rope(self.desc, self.kc, self.vc, slots.cuda(), pos.cuda(), self.dtable,
                               q, k, v, out)
        return out

    def logical(self, qkv, pos):
        """Rotated q, k as the cache's type holds them, and v, in fp64."""
        q, k, v = qkv.double().split([self.Hq, self.Hkv, self.Hkv], 1)
        return (rotate(q, self.table, pos, False).to(self.dt).double(),
                rotate(k, self.table, pos, False).to(self.dt).double(), v)

    def check(self, got, q, b, t, cap=0.0, slopes=None):
        ref, tol = attend(q, self.K[b], self.V[b], self.scale, t, cap, slopes)
        step = 2 * 2.0 ** (-7 if self.cache == "bf16" else -10) * \
            q.abs().amax() * self.K[b][:t + 1].abs().amax() * self.scale
        tol = tol + 2 * step * self.V[b].abs().amax()
        bound = tol[:, None] + half_step(ref.abs() + tol[:, None], "f32")
        assert ((got.double().cpu() - ref).abs() <= bound).all()


@pytest.mark.parametrize("cache,cap,use_slopes", [("bf16", 30.0, False), ("f16", 0.0, True),
                                                  ("bf16", 20.0, True)])
def test_chunked_prompt_then_decode_with_biased_scores(cache, cap, use_slopes):
    B, Hq, Hkv, d = 3, 8, 2, 128
    s = Server(B, Hq, Hkv, d, 64, cache, 14, seed=5)
    slopes = torch.tensor([0.01 * 2.0 ** -i for i in range(Hq)]) if use_slopes else None
    dslopes = None if slopes is None else slopes.cuda()
    lens = [0, 0, 0]
    for chunks in ([17, 100, 1], [60, 0, 33]):  # the prompts come in two calls
        total = sum(chunks)
        qkv = s.new(total, 3.0)
        pos = torch.cat([torch.arange(lens[b], lens[b] + n) for b, n in enumerate(chunks)])
        slots = torch.cat([s.slots(b, torch.arange(lens[b], lens[b] + n))
                           for b, n in enumerate(chunks)])
        q = s.append(qkv, slots, pos)
        lq, lk, lv = s.logical(qkv, pos)
        at = 0
        for b, n in enumerate(chunks):
            s.K[b] = torch.cat([s.K[b], lk[at:at + n]])
            s.V[b] = torch.cat([s.V[b], lv[at:at + n]])
            lens[b] += n
            at += n
        start = torch.tensor([0] + list(torch.tensor(chunks).cumsum(0)), dtype=torch.int32)
        out = torch.empty(total, Hq, d, device="cuda")
        pkv.pkv_paged_prefill_attention_biased(
            s.desc, q, s.kc, s.vc, s.dtables, torch.tensor(lens, dtype=torch.int32).cuda(),
            start.cuda(), max(chunks), s.scale, out, softcap=cap, alibi_slopes=dslopes)
        for b, n in enumerate(chunks):
            for j in {0, n // 2, n - 1} if n else ():
                i = int(start[b]) + j
                s.check(out[i], lq[i], b, lens[b] - n + j, cap, slopes)
    ws = torch.zeros(pkv.pkv_decode_workspace_bytes(s.desc, B, s.tables.shape[1]),
                     dtype=torch.uint8, device="cuda")
    for _ in range(18):  # over a page's end
        qkv = s.new(B, 3.0)
        pos = torch.tensor(lens)
        q = s.append(qkv, torch.cat([s.slots(b, pos[b:b + 1]) for b in range(B)]), pos)
        lq, lk, lv = s.logical(qkv, pos)
        for b in range(B):
            s.K[b], s.V[b] = torch.cat([s.K[b], lk[b:b + 1]]), torch.cat([s.V[b], lv[b:b + 1]])
            lens[b] += 1
        out = torch.empty(B, Hq, d, device="cuda")
        pkv.pkv_paged_decode_attention_biased(
            s.desc, q, s.kc, s.vc, s.dtables, torch.tensor(lens, dtype=torch.int32).cuda(),
            s.scale, out, ws, softcap=cap, alibi_slopes=dslopes)
        for b in range(B):
            s.check(out[b], lq[b], b, lens[b] - 1, cap, slopes)
    assert s.err.item() == 0


@pytest.mark.parametrize("prefix", [512, 4096])  # read for every sequence, and once
def test_steps_behind_a_shared_prompt_in_a_graph(prefix):
    """The prompt is appended once; then steps of append and shared-prefix decode
    replayed from one graph, whose inputs, slots and lengths change."""
    B, Hq, Hkv, d = 40, 8, 2, 128
    s = Server(B, Hq, Hkv, d, 128, "bf16", 4, prefix // PAGE, seed=6)
    qkv = s.new(prefix, 1.0)
    pos = torch.arange(prefix)
    s.append(qkv, s.slots(0, pos), pos)
    _, lk, lv = s.logical(qkv, pos)
    s.K, s.V = [lk] * B, [lv] * B
    lens = [prefix + b % 7 for b in range(B)]  # some have answers already
    for b in range(B):
        n = lens[b] - prefix
        if n:
            pos = torch.arange(prefix, lens[b])
            qkv = s.new(n, 1.0)
            s.append(qkv, s.slots(b, pos), pos)
            _, lk, lv = s.logical(qkv, pos)
            s.K[b], s.V[b] = torch.cat([s.K[b], lk]), torch.cat([s.V[b], lv])
    mbs = s.tables.shape[1]
    ws = torch.zeros(pkv.pkv_shared_prefix_workspace_bytes(s.desc, B, prefix // PAGE, mbs),
                     dtype=torch.uint8, device="cuda")
    qkv_d = torch.zeros(B, Hq + 2 * Hkv, d, dtype=s.dt, device="cuda")
    slots_d, pos_d = (torch.zeros(B, dtype=torch.int64, device="cuda") for _ in range(2))
    ctx_d = torch.zeros(B, dtype=torch.int32, device="cuda")
    pre_d = s.prefix.cuda()
    q_d = torch.empty(B, Hq, d, dtype=s.dt, device="cuda")
    out = torch.empty(B, Hq, d, device="cuda")

    def step():
        q, k, v = qkv_d.split([Hq, Hkv, Hkv], 1)
        pkv.pkv_kv_append_rope(s.desc, s.kc, s.vc, slots_d, pos_d, s.dtable, q, k, v, q_d)
        pkv.pkv_paged_decode_attention_shared_prefix(s.desc, q_d, s.kc, s.vc, pre_d, s.dtables,
                                                     ctx_d, s.scale, out, ws)

    graph = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    slots_d.fill_(-1)  # the captured step writes nothing by itself
    with torch.cuda.graph(graph, stream=st):
        step()
    for _ in range(20):
        qkv = s.new(B, 2.0)
        pos = torch.tensor(lens)
        qkv_d.copy_(qkv)
        pos_d.copy_(pos)
        slots_d.copy_(torch.cat([s.slots(b, pos[b:b + 1]) for b in range(B)]))
        lq, lk, lv = s.logical(qkv, pos)
        for b in range(B):
            s.K[b], s.V[b] = torch.cat([s.K[b], lk[b:b + 1]]), torch.cat([s.V[b], lv[b:b + 1]])
            lens[b] += 1
        ctx_d.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for b in (0, 1, 6, 13, 39):
            s.check(out[b], lq[b], b, lens[b] - 1)
    assert s.err.item() == 0
