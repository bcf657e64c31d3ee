"""Softmax weights far below the largest: a first token that takes nearly all the
weight and whose V is zero (an attention sink) in front of thousands of tokens that
weigh something only together.  What each of them weighs has to survive its rounding
to the 16-bit pair that the tensor cores multiply with V."""
import math

import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import CODE, DT, PAGE

pytestmark = pytest.mark.gpu

GAPS = (9.0, 14.0, 16.5, 17.4)  # nats between the first token's score and the others'


class Sink:
    """`batch` sequences of n tokens in the same blocks.  The token at `first` has a
    key of 8 in element 0 and no value; the others have no key and values around 1."""

    def __init__(self, n, batch, Hq, Hkv, d, cache, seed, first=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.batch, self.Hq, self.Hkv, self.d, self.first = n, batch, Hq, Hkv, d, first
        self.fp8 = cache.startswith("e4m3")
        pages = -(-n // PAGE)
        self.NB = pages + 2
        tables = torch.randperm(self.NB, generator=g)[:pages].to(torch.int32)
        blk, off = tables.long().repeat_interleave(PAGE)[:n], torch.arange(n) % PAGE
        v = 0.5 + torch.rand(n, Hkv, d, generator=g)
        v[first] = 0.0
        shape = (self.NB, Hkv, PAGE, d)
        ks = vs = None
        if self.fp8:  # codes of 256 v, scales of 1 / 256; the key a code of 256 under 1 / 32
            kc, vc = torch.zeros(shape, dtype=torch.uint8), torch.zeros(shape, dtype=torch.uint8)
            code = (v * 256).to(torch.float8_e4m3fn)
            vc[blk, :, off] = code.view(torch.uint8)
            self.V = code.double() / 256
            kc[blk[first], :, off[first], 0] = torch.tensor([256.0]).to(
                torch.float8_e4m3fn).view(torch.uint8)
            if cache == "e4m3":
                ks, vs = torch.full((Hkv,), 1 / 32), torch.full((Hkv,), 1 / 256)
            else:
                ks = torch.full((self.NB, Hkv, 2, PAGE), 1 / 256)
                ks[:, :, 0] = 1 / 32
        else:
            kc, vc = torch.zeros(shape, dtype=DT[cache]), torch.zeros(shape, dtype=DT[cache])
            v = v.to(DT[cache])
            vc[blk, :, off] = v
            self.V = v.double()
            kc[blk[first], :, off[first], 0] = 8.0
        self.qdt = DT.get(cache, torch.bfloat16)
        self.scale = 1 / math.sqrt(d)
        self.kc, self.vc = kc.cuda(), vc.cuda()
        self.ks, self.vs = (None if t is None else t.cuda() for t in (ks, vs))
        self.tables = tables.repeat(batch, 1).contiguous().cuda()
        self.blocks = tables.cuda()
        self.ctx = torch.full((batch,), n, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.desc = pkv.make_desc(self.NB, PAGE, Hkv, Hq, d, CODE[cache], self.ks, self.vs,
                                  self.err)

    def queries(self, rows, seed):
        """[rows][Hq][d]; the gaps in turn, row by row and head by head."""
        g = torch.Generator().manual_seed(seed)
        q = torch.randn(rows, self.Hq, self.d, generator=g)
        at = torch.arange(rows)[:, None] + torch.arange(self.Hq)[None, :]
        q[:, :, 0] = torch.tensor(GAPS)[at % len(GAPS)] / (8 * self.scale)
        return q.to(self.qdt)

    def check(self, out, q, seen, cap=0.0, slopes=None):
        """out, q: [rows][Hq][d]; row r sees the first seen[r] tokens.

        Off by, relative to the output: 2^-15 (pairs of bf16, exponentials, scores of
        up to 26 in log2 units), 2^-21 of a cap; n 2^-24 for sums of n terms in fp32,
        each cut at 2^-23 of the sum and 16 of them or more added at once.  And what
        the pairs cannot hold: half a step of an fp16 subnormal, 2^-25, of n weights
        that are kept 2^7 above their ratio to the largest."""
        ref = {}
        worst = 0.0
        for r in range(out.shape[0]):
            for h in range(self.Hq):
                x = float(q[r, h, 0])
                slope = 0.0 if slopes is None else float(slopes[h])
                kv = h // (self.Hq // self.Hkv)
                key = (x, slope, kv, seen[r])
                if key not in ref:
                    s = torch.zeros(seen[r], dtype=torch.float64)
                    s[self.first] = x * 8 * self.scale
                    if cap:
                        s = cap * torch.tanh(s / cap)
                    s += slope * (torch.arange(seen[r]).double() - (seen[r] - 1))
                    ref[key] = torch.softmax(s, 0) @ self.V[:seen[r], kv]
                want, n = ref[key], seen[r]
                tol = want.abs() * (2.0 ** -15 + cap * 2.0 ** -21 + n * 2.0 ** -24) + \
                    n * 2.0 ** -32 * 1.5
                off = (out[r, h] - want).abs()
                worst = max(worst, (off / tol).max().item())
        assert worst <= 1.0, f"{worst:.3g} of the bound"
        assert self.err.item() == 0


def zeros(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


# As many sequences as leave each of them whole, or nearly, to one share of the work.
@pytest.mark.parametrize("Hq,d,cache", [(1, 128, "f16"), (8, 64, "f16"), (4, 128, "bf16")])
@pytest.mark.parametrize("nodes", [1, 40])
def test_tree(Hq, d, cache, nodes):
    s = Sink(32768, 320, Hq, 1, d, cache, 11)
    q = s.queries(nodes, 12)
    total = 320 * nodes
    words = torch.tensor([1 << j for j in range(nodes)]).repeat(320).cuda()
    out = torch.empty(total, Hq, d, device="cuda")
    starts = (nodes * torch.arange(321)).int().cuda()
    pkv.pkv_paged_tree_attention(s.desc, q.repeat(320, 1, 1).cuda(), s.kc, s.vc, s.tables, s.ctx,
                                 starts, nodes, words, s.scale, out,
                                 zeros(pkv.pkv_tree_workspace_bytes(s.desc, 320, nodes, 2048)))
    out = out.view(320, nodes, Hq, d).double().cpu()
    # a node sees the past and itself: as if it came right behind the past
    see = [s.n - nodes + 1] * nodes
    V = s.V
    for b in (0, 1, 77, 200, 319):
        for j in range(0, nodes, 13):
            s.V = torch.cat([V[:s.n - nodes], V[s.n - nodes + j][None]])
            s.check(out[b, j:j + 1], q[j:j + 1], see[:1])
    s.V = V


def decode_out(s, q, call, **kw):
    out = torch.empty(q.shape, device="cuda")
    call(s.desc, q.cuda(), s.kc, s.vc, s.tables, s.ctx, out=out, scale=s.scale, **kw)
    return out.double().cpu()


CACHES = [("f16", 128, 1), ("f16", 64, 8), ("bf16", 128, 4), ("e4m3", 128, 4), ("e4m3tok", 128, 4),
          ("e4m3tok", 128, 1)]


@pytest.mark.parametrize("cache,d,Hq", CACHES)
@pytest.mark.parametrize("batch", [1, 320])
@pytest.mark.parametrize("form", ["plain", "scored", "cap", "distance"])
def test_decode(cache, d, Hq, batch, form):
    s = Sink(32768, batch, Hq, 1, d, cache, 21)
    q = s.queries(batch, 22)
    ws = zeros(pkv.pkv_decode_workspace_bytes(s.desc, batch, 2048))
    cap, slopes = 0.0, None
    if form == "plain":
        out = decode_out(s, q, pkv.pkv_paged_decode_attention, workspace=ws)
    elif form == "scored":
        ws = zeros(pkv.pkv_scored_workspace_bytes(s.desc, batch, 2048))
        out = decode_out(s, q, pkv.pkv_paged_decode_attention_scored, workspace=ws, decay=0.0,
                         weights=torch.zeros(s.NB, 1, PAGE, device="cuda"))
    else:
        cap = 50.0 if form == "cap" else 0.0
        slopes = torch.full((Hq,), 2.0 ** -16) if form == "distance" else None
        out = decode_out(s, q, pkv.pkv_paged_decode_attention_biased, workspace=ws, softcap=cap,
                         alibi_slopes=None if slopes is None else slopes.cuda())
    at = list(range(0, batch, 40))
    s.check(out[at], q[at], [s.n] * len(at), cap, slopes)


@pytest.mark.parametrize("cache,d,Hq", CACHES)
@pytest.mark.parametrize("batch", [1, 320])
@pytest.mark.parametrize("q_len", [2, 8])
def test_multi_query(cache, d, Hq, batch, q_len):
    s = Sink(32768, batch, Hq, 1, d, cache, 31)
    q = s.queries(batch * q_len, 32).view(batch, q_len, Hq, d)
    ws = zeros(pkv.pkv_decode_workspace_bytes_multi(s.desc, batch, q_len, 2048))
    out = decode_out(s, q, pkv.pkv_paged_decode_attention_multi, workspace=ws)
    for b in range(0, batch, 80):
        s.check(out[b], q[b], [s.n - q_len + j + 1 for j in range(q_len)])


@pytest.mark.parametrize("cache,d,Hq", CACHES[:3])
@pytest.mark.parametrize("form", ["plain", "cap", "distance", "both"])
def test_prefill(cache, d, Hq, form):
    rows = 40
    s = Sink(32768, 1, Hq, 1, d, cache, 51)
    q = s.queries(rows, 52)
    starts = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    kw, cap, slopes = {}, 0.0, None
    call = pkv.pkv_paged_prefill_attention
    if form != "plain":
        call = pkv.pkv_paged_prefill_attention_biased
        cap = 50.0 if form != "distance" else 0.0
        slopes = torch.full((Hq,), 2.0 ** -16) if form != "cap" else None
        kw = dict(softcap=cap, alibi_slopes=None if slopes is None else slopes.cuda())
    out = decode_out(s, q, call, q_start=starts, max_q_len=rows, **kw)
    s.check(out[::13], q[::13], [s.n - rows + j + 1 for j in range(0, rows, 13)], cap, slopes)


# The first token in the shared prefix, with and without a pass of its own for that
# (320 sequences and 2), and in what is each sequence's own (prefix of one block).
@pytest.mark.parametrize("cache,d,Hq", CACHES[:3])
@pytest.mark.parametrize("batch,prefix,first", [(320, 30000, 0), (2, 30000, 0), (320, 16, 16)])
def test_shared_prefix(cache, d, Hq, batch, prefix, first):
    s = Sink(32768, batch, Hq, 1, d, cache, 41, first)
    q = s.queries(batch, 42)
    npb = prefix // PAGE
    ws = zeros(pkv.pkv_shared_prefix_workspace_bytes(s.desc, batch, npb, 2048))
    out = torch.empty(q.shape, device="cuda")
    pkv.pkv_paged_decode_attention_shared_prefix(s.desc, q.cuda(), s.kc, s.vc,
                                                 s.blocks[:npb].contiguous(), s.tables, s.ctx,
                                                 s.scale, out, ws)
    at = list(range(0, batch, 40))
    s.check(out.double().cpu()[at], q[at], [s.n] * len(at))
