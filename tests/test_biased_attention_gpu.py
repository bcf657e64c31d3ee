"""Decode and prefill attention with scores capped by a tanh, with a distance
bias, and with both, against the formula in 64 bits."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import DT, Paged, alibi, attend, check

pytestmark = pytest.mark.gpu


def decode(p, q, out="f32", cap=0.0, slopes=None, window=0, sinks=0, ws=None):
    B = len(p.lens)
    if ws is None:
        ws = torch.zeros(pkv.pkv_decode_workspace_bytes(p.desc, B, p.mbs), dtype=torch.uint8,
                         device="cuda")
    o = torch.full((B, p.Hq, p.d), float("nan"), dtype=DT[out], device="cuda")
    pkv.pkv_paged_decode_attention_biased(
        p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, p.scale, o, ws, softcap=cap,
        alibi_slopes=None if slopes is None else slopes.cuda(), window=window, sinks=sinks)
    torch.cuda.synchronize()
    return o


def expect_decode(p, q, cap=0.0, slopes=None, window=0, sinks=0):
    rows = [attend(q[b].double(), p.K[b], p.V[b], p.scale, n - 1, cap, slopes, window, sinks)
            for b, n in enumerate(p.lens)]
    return torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows])


LENS = [1, 0, 15, 16, 17, 33, 700, 255, 1300]
DECODE = [  # Hq, Hkv, d, cache, cap, alibi, window, sinks, out, gain
    (8, 2, 128, "bf16", 30.0, False, 0, 0, "f32", 6.0),
    (8, 8, 64, "f16", 0.0, True, 0, 0, "f32", 1.0),
    (8, 1, 128, "f16", 5.0, True, 0, 0, "f16", 3.0),
    (6, 3, 128, "bf16", 50.0, True, 40, 0, "f32", 6.0),
    (4, 1, 64, "bf16", 50.0, False, 1, 0, "bf16", 2.0),
    (4, 4, 64, "f16", 0.0, True, 100, 5, "f32", 1.0),
    (8, 2, 128, "e4m3", 30.0, True, 0, 0, "f32", 6.0),
    (8, 1, 128, "e4m3", 20.0, False, 64, 3, "bf16", 4.0),
    (8, 2, 128, "e4m3tok", 30.0, False, 0, 0, "f32", 6.0),
    (4, 4, 128, "e4m3tok", 0.0, True, 200, 20, "f32", 1.0),
    (8, 2, 128, "bf16", 1000.0, False, 0, 0, "f32", 6.0),
    (8, 2, 128, "bf16", 2.0 ** -10, False, 0, 0, "f32", 6.0),
    (8, 2, 128, "bf16", 2.0 ** 10, False, 0, 0, "f32", 1.0),
]


def e4m3_slack(p, q):
    """bf16 q meets an E4M3 cache in fp16, at most half an fp16 step (2^-11)
    of each of its elements off where bf16 has more range than fp16: none at
    these magnitudes (bf16 has fewer bits), so nothing to add."""
    return 0.0


@pytest.mark.parametrize("case", DECODE)
def test_decode_matches_the_formula(case):
    Hq, Hkv, d, cache, cap, use_slopes, window, sinks, out, gain = case
    p = Paged(LENS, Hq, Hkv, d, cache, 11)
    q = p.queries(len(LENS), 12, gain)
    sl = alibi(Hq) if use_slopes else None
    o = decode(p, q, out, cap, sl, window, sinks)
    assert p.err.item() == 0
    ref, tol = expect_decode(p, q, cap, sl, window, sinks)
    check(o, ref, tol + e4m3_slack(p, q), out, str(case))
    assert torch.all(o[1] == 0)  # the empty sequence


@pytest.mark.parametrize("cap,use_slopes", [(30.0, False), (0.0, True), (30.0, True)])
def test_decode_long_context_over_many_shares(cap, use_slopes):
    """One sequence of 20000 tokens cut over many CTAs beside a short one; the
    same bits again on a second call."""
    p = Paged([20000, 3], 4, 1, 128, "bf16", 13)
    q = p.queries(2, 14, 4.0)
    sl = alibi(4) if use_slopes else None
    o = decode(p, q, "f32", cap, sl)
    ref, tol = expect_decode(p, q, cap, sl)
    check(o, ref, tol, "f32")
    assert torch.equal(o, decode(p, q, "f32", cap, sl))


def test_slopes_of_any_sign():
    p = Paged([300, 90], 4, 2, 64, "f16", 15)
    q = p.queries(2, 16)
    sl = torch.tensor([-0.02, 0.0, 3.0, -0.5])
    ref, tol = expect_decode(p, q, 0.0, sl)
    check(decode(p, q, "f32", 0.0, sl), ref, tol, "f32")


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_with_neither_it_is_the_plain_call(cache):
    p = Paged(LENS, 8, 2, 128, cache, 17)
    q = p.queries(len(LENS), 18)
    ws = torch.zeros(pkv.pkv_decode_workspace_bytes(p.desc, len(LENS), p.mbs), dtype=torch.uint8,
                     device="cuda")
    a = decode(p, q, ws=ws)
    b = torch.empty_like(a)
    pkv.pkv_paged_decode_attention(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, p.scale, b, ws)
    assert torch.equal(a, b)
    # slopes of zero change no score
    check(decode(p, q, "f32", 0.0, torch.zeros(8)), b.double().cpu(),
          torch.full((len(LENS), 8), 1e-5, dtype=torch.float64), "f32")


def test_bad_blocks_and_lengths_are_reported():
    p = Paged([40, 60], 8, 2, 128, "bf16", 19)
    q = p.queries(2, 20)
    p.tables[0, 1] = 10 ** 8
    o = decode(p, q, "f32", 30.0, alibi(8))
    assert p.err.item() == pkv.PKV_ERR_BOUNDS
    ref, tol = expect_decode(p, q, 30.0, alibi(8))
    check(o[1:], ref[1:], tol[1:], "f32")
    p.err.zero_()
    p.ctx[1] = p.mbs * 16 + 1
    o = decode(p, q, "f32", 30.0, alibi(8))
    assert p.err.item() == pkv.PKV_ERR_BOUNDS
    assert torch.all(o[1] == 0)


@pytest.mark.parametrize("n", [40, 3000])
def test_nan_shows_where_it_is_seen(n):
    """A NaN in a key reaches every output of its sequence and KV head, whether
    or not the sequence is cut over several CTAs, and nothing else."""
    p = Paged([n, 200, n], 4, 2, 128, "bf16", 91)
    q = p.queries(3, 92, 2.0)
    p.kc[int(p.tables[0, n // 32]), 1, 2, 5] = float("nan")
    o = decode(p, q, "f32", 30.0, alibi(4))
    assert torch.isnan(o[0, 2:]).all()
    ref, tol = expect_decode(p, q, 30.0, alibi(4))
    check(o[1:], ref[1:], tol[1:], "f32")
    check(o[0, :2], ref[0, :2], tol[0, :2], "f32")


# ---------------------------------------------------------------- prefill
def prefill(p, q, chunks, out="f32", cap=0.0, slopes=None, total=None):
    st = torch.tensor([0] + list(torch.tensor(chunks).cumsum(0)), dtype=torch.int32)
    o = torch.full(q.shape, 7.0, dtype=DT[out], device="cuda")
    pkv.pkv_paged_prefill_attention_biased(
        p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, st.cuda(), max(chunks), p.scale, o,
        softcap=cap, alibi_slopes=None if slopes is None else slopes.cuda())
    torch.cuda.synchronize()
    return o


def expect_prefill(p, q, chunks, cap, slopes):
    rows, at = [], 0
    for b, n in enumerate(chunks):
        for j in range(n):
            rows.append(attend(q[at + j].double(), p.K[b], p.V[b], p.scale,
                               p.lens[b] - n + j, cap, slopes))
        at += n
    return torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows])


PREFILL = [  # Hq, Hkv, d, cache, lens, chunks, cap, alibi, out, gain
    (4, 1, 64, "f16", [1, 17, 300], [1, 17, 130], 0.0, True, "f32", 1.0),
    (4, 4, 128, "bf16", [40, 333, 128], [40, 60, 0], 30.0, False, "f32", 6.0),
    (8, 1, 128, "f16", [200, 129], [33, 129], 5.0, True, "f16", 3.0),
    (2, 1, 128, "bf16", [700, 16], [200, 5], 50.0, True, "bf16", 6.0),
    (4, 2, 64, "bf16", [260, 64], [130, 1], 300.0, False, "f32", 6.0),
    (4, 2, 64, "f16", [260, 64], [130, 1], 300.0, True, "f32", 6.0),
    (4, 2, 128, "bf16", [150, 64], [100, 64], 2.0 ** 10, False, "f32", 1.0),
]


@pytest.mark.parametrize("case", PREFILL)
def test_prefill_matches_the_formula(case):
    Hq, Hkv, d, cache, lens, chunks, cap, use_slopes, out, gain = case
    p = Paged(lens, Hq, Hkv, d, cache, 23)
    q = p.queries(sum(chunks) + 3, 24, gain)  # three rows behind the last sequence
    sl = alibi(Hq) if use_slopes else None
    o = prefill(p, q, chunks, out, cap, sl)
    assert p.err.item() == 0
    ref, tol = expect_prefill(p, q, chunks, cap, sl)
    check(o[:sum(chunks)], ref, tol, out, str(case))
    assert torch.all(o[sum(chunks):] == 7.0)  # left as they were


@pytest.mark.parametrize("cache", ["bf16", "f16"])
@pytest.mark.parametrize("slopes", [(3.0, -4.0, 0.001, 40.0), (2.0, -2.0, 1.8, -1.8)])
def test_prefill_cap_with_slopes_of_any_size(cache, slopes):
    """Slopes so steep that a reference maximum a few tokens off would lose the
    weights, of either sign, and just below that."""
    p = Paged([300, 140, 37], 4, 2, 64, cache, 93)
    chunks = [150, 140, 2]
    q = p.queries(sum(chunks), 94, 3.0)
    sl = torch.tensor(slopes)
    o = prefill(p, q, chunks, "f32", 20.0, sl)
    ref, tol = expect_prefill(p, q, chunks, 20.0, sl)
    check(o, ref, tol, "f32", str(slopes))


@pytest.mark.parametrize("cap,use_slopes", [(30.0, False), (0.0, True)])
def test_prefill_long_sampled(cap, use_slopes):
    """600 rows behind 2500 cached tokens, sampled rows."""
    p = Paged([3100], 8, 2, 128, "bf16", 25)
    q = p.queries(600, 26, 4.0)
    sl = alibi(8) if use_slopes else None
    o = prefill(p, q, [600], "f32", cap, sl)
    for j in (0, 127, 128, 255, 256, 511, 599):
        ref, tol = attend(q[j].double(), p.K[0], p.V[0], p.scale, 2500 + j, cap, sl)
        check(o[j], ref, tol, "f32", f"row {j}")
    assert torch.equal(o, prefill(p, q, [600], "f32", cap, sl))


def test_prefill_with_neither_is_the_plain_call():
    p = Paged([300, 50], 8, 2, 128, "bf16", 27)
    q = p.queries(150, 28)
    a = prefill(p, q, [100, 50])
    b = torch.empty_like(a)
    st = torch.tensor([0, 100, 150], dtype=torch.int32, device="cuda")
    pkv.pkv_paged_prefill_attention(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, st, 100,
                                    p.scale, b)
    assert torch.equal(a, b)


def test_one_row_prefill_and_decode_agree():
    p = Paged([1, 33, 900], 8, 2, 128, "bf16", 29)
    q = p.queries(3, 30, 4.0)
    sl = alibi(8)
    ref, tol = expect_decode(p, q, 20.0, sl)
    check(prefill(p, q, [1, 1, 1], "f32", 20.0, sl), ref, tol, "f32")
    check(decode(p, q, "f32", 20.0, sl), ref, tol, "f32")
