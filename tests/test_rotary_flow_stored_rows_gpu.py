"""Append, prefill and decode one after the other, held to the attention calls' own
error: the reference attends, in fp64, over the rows that the append stored, which
are first held to the rotation's own rounding."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import PAGE, attend, check, half_step, rotate
from test_rotary_decode_flow_gpu import Server

pytestmark = pytest.mark.gpu


class Stored(Server):
    def take(self, qkv, q_out, parts):
        """parts: (sequence, positions) of the rows of qkv, in order, as appended.
        Extends the logical rows by what the pool holds, after a look at each."""
        name = self.cache
        pos = torch.cat([x for _, x in parts])
        q, k, v = qkv.double().split([self.Hq, self.Hkv, self.Hkv], 1)
        got_q = q_out.double().cpu()
        at, rows_k, rows_v = 0, [], []
        for b, x in parts:
            slot = self.slots(b, x).cuda()
            rows_k.append(self.kc[slot // PAGE, :, slot % PAGE].double().cpu())
            rows_v.append(self.vc[slot // PAGE, :, slot % PAGE].double().cpu())
        got_k, got_v = torch.cat(rows_k), torch.cat(rows_v)
        for got, src in ((got_q, q), (got_k, k)):
            # two products and a sum in fp32, then half a step of the type
            arith = 2.0 ** -22 * src.abs().amax(-1, keepdim=True)
            y = rotate(src, self.table, pos, False)
            assert ((got - y).abs() <= half_step(y.abs() + arith, name) + arith).all()
        assert torch.equal(got_v, v)
        for b, x in parts:
            n = len(x)
            self.K[b] = torch.cat([self.K[b], got_k[at:at + n]])
            self.V[b] = torch.cat([self.V[b], got_v[at:at + n]])
            at += n
        return got_q

    def hold(self, out, q, b, t, cap=0.0, slopes=None, what=""):
        ref, tol = attend(q, self.K[b], self.V[b], self.scale, t, cap, slopes)
        check(out, ref, tol, "f32", what)


@pytest.mark.parametrize("cache,cap,use_slopes,rot", [
    ("bf16", 30.0, False, 64), ("f16", 0.0, True, 128), ("bf16", 20.0, True, 128),
    ("f16", 50.0, False, 32)])
def test_prompts_in_chunks_then_steps(cache, cap, use_slopes, rot):
    B, Hq, Hkv, d = 4, 8, 2, 128
    s = Stored(B, Hq, Hkv, d, rot, cache, 16, seed=15)
    sl = torch.tensor([0.02 * 2.0 ** -i for i in range(Hq)]) if use_slopes else None
    dsl = None if sl is None else sl.cuda()
    lens = [0] * B
    for chunks in ([17, 130, 1, 64], [60, 0, 33, 65]):
        parts = [(b, torch.arange(lens[b], lens[b] + n)) for b, n in enumerate(chunks)]
        pos = torch.cat([x for _, x in parts])
        qkv = s.new(sum(chunks), 3.0)
        q = s.append(qkv, torch.cat([s.slots(b, x) for b, x in parts]), pos)
        hq = s.take(qkv, q, parts)
        lens = [a + n for a, n in zip(lens, chunks)]
        start = torch.tensor([0] + list(torch.tensor(chunks).cumsum(0)), dtype=torch.int32)
        out = torch.empty(sum(chunks), Hq, d, device="cuda")
        pkv.pkv_paged_prefill_attention_biased(
            s.desc, q, s.kc, s.vc, s.dtables, torch.tensor(lens, dtype=torch.int32).cuda(),
            start.cuda(), max(chunks), s.scale, out, softcap=cap, alibi_slopes=dsl)
        for b, n in enumerate(chunks):
            for j in {0, n // 2, n - 1} if n else ():
                i = int(start[b]) + j
                s.hold(out[i], hq[i], b, lens[b] - n + j, cap, sl, f"prompt {b} row {j}")
    ws = torch.zeros(pkv.pkv_decode_workspace_bytes(s.desc, B, s.tables.shape[1]),
                     dtype=torch.uint8, device="cuda")
    for step in range(18):  # over a page's end
        parts = [(b, torch.tensor([lens[b]])) for b in range(B)]
        qkv = s.new(B, 3.0)
        q = s.append(qkv, torch.cat([s.slots(b, x) for b, x in parts]), torch.tensor(lens))
        hq = s.take(qkv, q, parts)
        lens = [n + 1 for n in lens]
        out = torch.empty(B, Hq, d, device="cuda")
        pkv.pkv_paged_decode_attention_biased(
            s.desc, q, s.kc, s.vc, s.dtables, torch.tensor(lens, dtype=torch.int32).cuda(),
            s.scale, out, ws, softcap=cap, alibi_slopes=dsl)
        for b in range(B):
            s.hold(out[b], hq[b], b, lens[b] - 1, cap, sl, f"step {step} sequence {b}")
    assert s.err.item() == 0


@pytest.mark.parametrize("prefix", [512, 4096])  # read for every sequence, and once
def test_steps_behind_a_shared_prompt(prefix):
    B, Hq, Hkv, d = 40, 8, 2, 128
    s = Stored(B, Hq, Hkv, d, 128, "bf16", 4, prefix // PAGE, seed=16)
    pos = torch.arange(prefix)
    qkv = s.new(prefix, 1.0)
    s.take(qkv, s.append(qkv, s.slots(0, pos), pos), [(0, pos)])
    s.K, s.V = [s.K[0]] * B, [s.V[0]] * B
    lens = [prefix] * B
    mbs = s.tables.shape[1]
    ws = torch.zeros(pkv.pkv_shared_prefix_workspace_bytes(s.desc, B, prefix // PAGE, mbs),
                     dtype=torch.uint8, device="cuda")
    pre = s.prefix.cuda()
    for step in range(20):
        parts = [(b, torch.tensor([lens[b]])) for b in range(B)]
        qkv = s.new(B, 2.0)
        q = s.append(qkv, torch.cat([s.slots(b, x) for b, x in parts]), torch.tensor(lens))
        hq = s.take(qkv, q, parts)
        lens = [n + 1 for n in lens]
        out = torch.empty(B, Hq, d, device="cuda")
        pkv.pkv_paged_decode_attention_shared_prefix(
            s.desc, q, s.kc, s.vc, pre, s.dtables, torch.tensor(lens, dtype=torch.int32).cuda(),
            s.scale, out, ws)
        for b in (0, 1, 6, 13, 39):
            s.hold(out[b], hq[b], b, lens[b] - 1, what=f"step {step} sequence {b}")
    assert s.err.item() == 0
