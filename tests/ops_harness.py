"""Inputs and 64-bit references for the rotary append, the shared-prefix decode
and the biased attention calls.

The pool is built from logical K and V rows; every slot that no sequence owns
holds NaN.  References are written from the formulas, in fp64, from the logical
rows alone (E4M3 rows as the stored codes stand for them)."""
from __future__ import annotations

import math

import numpy as np
import torch

import paged_kv_cache_250_gb300 as pkv

PAGE = 16
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"f16": pkv.PKV_F16, "bf16": pkv.PKV_BF16, "e4m3": pkv.PKV_FP8_E4M3,
        "e4m3tok": pkv.PKV_FP8_E4M3_TOKEN}


def half_step(x, name):
    """Half a step of the type at |x| (fp64 tensor)."""
    mant, emin = {"f16": (10, -14), "bf16": (7, -126), "f32": (23, -126),
                  "e4m3": (3, -6)}[name]
    e = torch.floor(torch.log2(x.abs().clamp_min(1e-300))).clamp_min(emin)
    return 0.5 * torch.exp2(e - mant)


class Paged:
    """K, V: lists of [n_b][Hkv][d] fp32 logical rows; prefix rows (shared by
    all sequences) come first in every sequence when `prefix` > 0 tokens."""

    def __init__(self, lens, Hq, Hkv, d, cache, seed, prefix=0, device="cuda", garbage_prefix=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hq, self.Hkv, self.d, self.cache = lens, Hq, Hkv, d, cache
        self.prefix = prefix
        assert prefix % PAGE == 0
        npb = prefix // PAGE
        own = [max(0, -(-n // PAGE) - npb) for n in lens]
        self.mbs = max(1, npb + max(own + [0]))
        NB = npb + sum(own) + 4
        perm = torch.randperm(NB, generator=g).tolist()
        self.NB = NB
        pre, at = perm[:npb], npb
        tables = torch.full((len(lens), self.mbs), -7, dtype=torch.int32)
        nan8 = 0x7F
        fp8 = cache.startswith("e4m3")
        kc = torch.full((NB, Hkv, PAGE, d), nan8 if fp8 else float("nan"),
                        dtype=torch.uint8 if fp8 else DT[cache])
        vc = kc.clone()
        self.ks = self.vs = None
        if cache == "e4m3":
            self.ks = (0.5 + torch.rand(Hkv, generator=g)) / 100
            self.vs = (0.5 + torch.rand(Hkv, generator=g)) / 100
        elif cache == "e4m3tok":
            self.ks = torch.full((NB, Hkv, 2, PAGE), float("nan"))

        def put(pages, n):  # n tokens into the pages: their logical values in fp64
            pair = []
            for i, c in enumerate((kc, vc)):
                x = torch.randn(n, Hkv, d, generator=g)
                blk = torch.tensor(pages, dtype=torch.long).repeat_interleave(PAGE)[:n]
                off = torch.arange(n) % PAGE
                if not fp8:
                    x = x.to(c.dtype)
                    c[blk, :, off] = x
                    pair.append(x.double())
                    continue
                if cache == "e4m3":
                    s = (self.ks if i == 0 else self.vs)[None, :].expand(n, Hkv)
                else:
                    s = x.abs().amax(-1) / 448
                    self.ks[blk, :, i, off] = s
                code = (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
                c[blk, :, off] = code.view(torch.uint8)
                pair.append(code.double() * s.double()[..., None])
            return pair

        seen = min(prefix, max(lens + [0]))
        self.pK, self.pV = put(pre, seen)
        self.K, self.V = [], []
        for b, n in enumerate(lens):
            if not garbage_prefix:
                tables[b, :npb] = torch.tensor(pre, dtype=torch.int32)
            tables[b, npb:npb + own[b]] = torch.tensor(perm[at:at + own[b]], dtype=torch.int32)
            k, v = put(perm[at:at + own[b]], max(0, n - prefix))
            at += own[b]
            self.K.append(torch.cat([self.pK[:min(n, prefix)], k]))
            self.V.append(torch.cat([self.pV[:min(n, prefix)], v]))
        self.dev = torch.device(device)
        put_dev = lambda t: None if t is None else t.to(self.dev).contiguous()  # noqa: E731
        self.kc, self.vc, self.tables = put_dev(kc), put_dev(vc), put_dev(tables)
        self.ks, self.vs = put_dev(self.ks), put_dev(self.vs)
        self.prefix_blocks = put_dev(torch.tensor(pre, dtype=torch.int32))
        self.ctx = put_dev(torch.tensor(lens, dtype=torch.int32))
        self.err = torch.zeros(1, dtype=torch.int32, device=self.dev)
        self.desc = pkv.make_desc(NB, PAGE, Hkv, Hq, d, CODE[cache], self.ks, self.vs, self.err)
        self.scale = 1.0 / math.sqrt(d)
        self.qdt = DT.get(cache, torch.bfloat16)

    def queries(self, rows, seed, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        return (gain * torch.randn(rows, self.Hq, self.d, generator=g)).to(self.qdt)


def attend(q, K, V, scale, t, cap=0.0, slopes=None, window=0, sinks=0):
    """One query row [Hq][d] at position t over rows 0 .. t of K, V
    [n][Hkv][d], all fp64; with it the error an fp32-accumulating kernel may
    make (see tolerance)."""
    Hq, d = q.shape
    Hkv = V.shape[1]
    out = torch.zeros(Hq, d, dtype=torch.float64)
    tol = torch.zeros(Hq, dtype=torch.float64)
    if t < 0:
        return out, tol
    u = torch.arange(t + 1)
    keep = torch.ones(t + 1, dtype=torch.bool)
    if window > 0:
        keep = (u > t - window) | (u < sinks)
    u = u[keep]
    for h in range(Hq):
        k, v = K[u, h // (Hq // Hkv)], V[u, h // (Hq // Hkv)]
        s = (k @ q[h]) * scale
        size = (k.abs() @ q[h].abs() * abs(scale)).max()
        bias = 0.0
        if cap > 0:
            s = cap * torch.tanh(s / cap)
        if slopes is not None:
            b = float(slopes[h]) * (u - t).double()
            s = s + b
            near = s > s.max() - 40  # the others weigh e^-40 at most
            bias = max(b[near].abs().max().item(), s[near].abs().max().item())
        p = torch.exp(s - s.max())
        out[h] = (p[:, None] * v).sum(0) / p.sum()
        # Score error: d products summed in fp32, each addition cut (not
        # rounded) at 2^-23 of sums that stay below `size`; 2^-21 of the
        # cap (the tanh's 2^-22 and its scaling); 20 roundings of the bias.
        # A weight's own error: 2^-16 (its 16-bit pair), 2^-21 (exp2).
        ds = size * d * 2.0 ** -23 + cap * 2.0 ** -21 + bias * 20 * 2.0 ** -24
        tol[h] = v.abs().max() * 2 * (ds + 2.0 ** -15)
    return out, tol


def check(got, ref, tol, out_type, what=""):
    got, ref = got.double().cpu(), ref
    bound = tol[..., None] + half_step(ref.abs() + tol[..., None], out_type)
    off = (got - ref).abs()
    assert torch.isfinite(got).all(), what
    worst = (off / bound).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound, {off.max().item():.3g} off"


def alibi(Hq):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / Hq) for i in range(Hq)], dtype=torch.float32)


def rope_table(positions, rot, seed=None):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate(x, table, pos, interleaved):
    """x [T][H][d] fp64, the rows of table at pos."""
    rot = table.shape[1]
    cs = table.double()[pos]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def np64(t):
    return t.double().cpu().numpy().astype(np.float64)
