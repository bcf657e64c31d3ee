"""Workloads of the paged-cache operators: the rotary append, decode attention
over a shared prefix, and attention with capped or distance-biased scores.

``own`` chooses between the plain form (elementary torch operations in 32
bits) and the library's kernels.  A case is a dict of plain values;
``prepare`` draws its inputs on the GPU from a seed, ``run`` makes one pass.
"""
import math

import torch

own = False

PAGE = 16
DEVICE = "cuda"
_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _pkv():
    import paged_kv_cache_250_gb300 as pkv
    return pkv


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence: the append of a chat with one user, where latency counts
        {"name": "append_rope_1_token", "op": "append", "tokens": 1, "q_heads": 32, "kv_heads": 8,
         "d": 128, "rot": 128, "interleaved": False, "cache": "bf16", "max_pos": 8192},
        # a decode step of a server with an E4M3 cache, one scale per token
        {"name": "append_rope_batch_e4m3tok", "op": "append", "tokens": 96, "q_heads": 32,
         "kv_heads": 8, "d": 128, "rot": 128, "interleaved": False, "cache": "e4m3tok",
         "max_pos": 32768},
        # a prompt chunk over many sequences
        {"name": "append_rope_prompt", "op": "append", "tokens": 8192, "q_heads": 64,
         "kv_heads": 8, "d": 128, "rot": 128, "interleaved": False, "cache": "bf16",
         "max_pos": 32768},
        # a few requests behind a short system prompt, one KV head per query head, odd sizes
        {"name": "shared_prefix_small", "op": "shared", "batch": 5, "q_heads": 8, "kv_heads": 8,
         "d": 64, "cache": "f16", "prefix": 1040, "lo": 1, "hi": 77},
        # a serving batch behind a long system prompt, answers of up to 512 tokens
        {"name": "shared_prefix_batch", "op": "shared", "batch": 64, "q_heads": 32, "kv_heads": 8,
         "d": 128, "cache": "bf16", "prefix": 8192, "lo": 1, "hi": 512},
        # many samples of one long document
        {"name": "shared_prefix_many", "op": "shared", "batch": 256, "q_heads": 32, "kv_heads": 8,
         "d": 128, "cache": "bf16", "prefix": 32768, "lo": 1, "hi": 512},
        # one sequence, distance bias, odd length
        {"name": "biased_decode_1", "op": "decode", "batch": 1, "q_heads": 32, "kv_heads": 32,
         "d": 128, "cache": "f16", "lo": 701, "hi": 701, "cap": 0.0, "alibi": True, "window": 0},
        # a serving batch of ragged lengths, capped scores
        {"name": "biased_decode_batch", "op": "decode", "batch": 32, "q_heads": 32, "kv_heads": 8,
         "d": 128, "cache": "bf16", "lo": 1, "hi": 8192, "cap": 30.0, "alibi": False, "window": 0},
        # a windowed layer over an E4M3 cache, capped scores and distance bias
        {"name": "biased_decode_window_e4m3", "op": "decode", "batch": 64, "q_heads": 32,
         "kv_heads": 8, "d": 128, "cache": "e4m3", "lo": 500, "hi": 8192, "cap": 30.0,
         "alibi": True, "window": 4096},
        # a short prompt after a cached beginning, distance bias, odd sizes
        {"name": "biased_prefill_short", "op": "prefill", "batch": 1, "q_heads": 4, "kv_heads": 1,
         "d": 64, "cache": "f16", "chunk_lo": 201, "chunk_hi": 201, "past_lo": 133,
         "past_hi": 133, "cap": 0.0, "alibi": True},
        # ragged prompts of a continuous batch, eight query heads per KV head
        {"name": "biased_prefill_ragged", "op": "prefill", "batch": 12, "q_heads": 32,
         "kv_heads": 4, "d": 128, "cache": "bf16", "chunk_lo": 1, "chunk_hi": 700, "past_lo": 0,
         "past_hi": 1500, "cap": 50.0, "alibi": True},
        # long prompts in chunks
        {"name": "biased_prefill_long", "op": "prefill", "batch": 4, "q_heads": 32, "kv_heads": 8,
         "d": 128, "cache": "bf16", "chunk_lo": 2048, "chunk_hi": 2048, "past_lo": 6144,
         "past_hi": 6144, "cap": 30.0, "alibi": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    g = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 3, 4, 8])
    return g * hkv, hkv


def draw(rng):
    op = rng.choice(["append", "shared", "decode", "prefill"])
    hq, hkv = _heads(rng)
    d = rng.choice([64, 128, 128])
    if op == "append":
        cache = rng.choice(["f16", "bf16", "e4m3", "e4m3tok"])
        d = 128 if cache.startswith("e4m3") else d
        rot = rng.choice([d, d, d // 2, d // 4])
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "q_heads": hq, "kv_heads": hkv,
                "d": d, "rot": rot, "interleaved": rng.random() < 0.3, "cache": cache,
                "max_pos": _log_int(rng, 8192, 131072)}
    if op == "shared":
        hi = _log_int(rng, 1, 512)
        return {"op": op, "batch": _log_int(rng, 1, 256), "q_heads": min(hq, 32) // hkv * hkv,
                "kv_heads": hkv, "d": d, "cache": rng.choice(["f16", "bf16"]),
                "prefix": PAGE * _log_int(rng, 4, 2048), "lo": _log_int(rng, 1, hi), "hi": hi}
    if op == "decode":
        cache = rng.choice(["f16", "bf16", "e4m3", "e4m3tok"])
        d = 128 if cache.startswith("e4m3") else d
        kind = rng.choice([(30.0, False), (50.0, False), (0.0, True), (20.0, True)])
        hi = _log_int(rng, 1, 8192)
        return {"op": op, "batch": _log_int(rng, 1, 32), "q_heads": hq, "kv_heads": hkv, "d": d,
                "cache": cache, "lo": _log_int(rng, 1, hi), "hi": hi, "cap": kind[0],
                "alibi": kind[1], "window": rng.choice([0, 0, _log_int(rng, 1, 4096)])}
    kind = rng.choice([(30.0, False), (50.0, False), (0.0, True), (20.0, True)])
    chunk, past = _log_int(rng, 1, 2048), _log_int(rng, 1, 6145) - 1
    return {"op": op, "batch": _log_int(rng, 1, 4), "q_heads": min(hq, 32) // hkv * hkv,
            "kv_heads": hkv, "d": d, "cache": rng.choice(["f16", "bf16"]),
            "chunk_lo": _log_int(rng, 1, chunk), "chunk_hi": chunk, "past_lo": past // 2,
            "past_hi": past, "cap": kind[0], "alibi": kind[1]}


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], the same for every seed."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _visible(c):
    """Scores of one head: the (row, position) pairs that a pass looks at."""
    if c["op"] == "shared":
        return sum(c["prefix"] + s for s in _spread(c["lo"], c["hi"], c["batch"]))
    if c["op"] == "decode":
        return sum(min(n, c["window"]) if c["window"] else n
                   for n in _spread(c["lo"], c["hi"], c["batch"]))
    chunks = _spread(c["chunk_lo"], c["chunk_hi"], c["batch"])
    pasts = _spread(c["past_lo"], c["past_hi"], c["batch"])
    return sum(n * p + n * (n + 1) // 2 for n, p in zip(chunks, pasts))


def work(case):
    c = case
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["d"]
    e = 1 if c["cache"].startswith("e4m3") else 2
    tok = 8 if c["cache"] == "e4m3tok" else 0  # a token's two scales, per KV head
    if c["op"] == "append":
        t = c["tokens"]
        read = t * ((hq + 2 * hkv) * d * 2 + c["rot"] * 4 + 16)
        write = t * (hq * d * 2 + hkv * (2 * d * e + tok))
        return {"bytes": read + write, "flops": 3 * t * (hq + hkv) * c["rot"]}
    flops = 4 * d * hq * _visible(c)
    if c["op"] == "shared":
        own_tokens = sum(_spread(c["lo"], c["hi"], c["batch"]))
        kv = (c["prefix"] + own_tokens) * hkv * 2 * d * e
        rows = c["batch"]
        tables = 4 * (c["prefix"] // PAGE + sum(-(-s // PAGE) for s in
                                                 _spread(c["lo"], c["hi"], c["batch"])))
    elif c["op"] == "decode":
        kv = _visible(c) * hkv * (2 * d * e + tok)
        rows = c["batch"]
        tables = 4 * (_visible(c) // PAGE + c["batch"])
    else:
        chunks = _spread(c["chunk_lo"], c["chunk_hi"], c["batch"])
        pasts = _spread(c["past_lo"], c["past_hi"], c["batch"])
        kv = sum(n + p for n, p in zip(chunks, pasts)) * hkv * 2 * d * e
        rows = sum(chunks)
        tables = 4 * sum(-(-(n + p) // PAGE) for n, p in zip(chunks, pasts))
    return {"bytes": kv + rows * hq * d * 4 + tables + 4 * c["batch"], "flops": flops}


# ---------------------------------------------------------------- inputs
class State:
    pass


def _pool(s, c, blocks, g):
    """The two caches, [blocks][kv_heads][16][d], and their scales."""
    shape = (blocks, c["kv_heads"], PAGE, c["d"])
    s.ks = s.vs = None

    def filled():
        if c["cache"].startswith("e4m3"):
            x = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)
            return (x * 90.0).clamp(-448, 448).to(torch.float8_e4m3fn)
        return torch.randn(shape, generator=g, device=DEVICE, dtype=_DT[c["cache"]])

    s.kc, s.vc = filled(), filled()
    if c["cache"] == "e4m3":  # one scale per KV head, for K and for V
        s.ks = (0.5 + torch.rand(c["kv_heads"], generator=g, device=DEVICE)) / 90.0
        s.vs = (0.5 + torch.rand(c["kv_heads"], generator=g, device=DEVICE)) / 90.0
    elif c["cache"] == "e4m3tok":  # the pool of one scale per row: K's 16, then V's 16, a page
        s.ks = (0.5 + torch.rand((blocks, c["kv_heads"], 2, PAGE), generator=g,
                                 device=DEVICE)) / 90.0


def _alibi(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], dtype=torch.float32,
                        device=DEVICE)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE).manual_seed(1_000_003 * (int(seed) % 1_000_003) + 17)
    s = State()
    s.c = c
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["d"]
    dt = _DT.get(c["cache"], torch.bfloat16)
    s.scale = 1.0 / math.sqrt(d)
    s.dt = dt
    if c["op"] == "append":
        t = c["tokens"]
        blocks = (2 * t + PAGE - 1) // PAGE + 4
        _pool(s, c, blocks, g)
        # the projection's output: q, k and v beside one another in one row per token
        s.qkv = torch.randn((t, hq + 2 * hkv, d), generator=g, device=DEVICE).to(dt)
        s.q, s.k, s.v = s.qkv[:, :hq], s.qkv[:, hq:hq + hkv], s.qkv[:, hq + hkv:]
        s.slots = torch.randperm(blocks * PAGE, generator=g, device=DEVICE)[:t].contiguous()
        s.pos = torch.randint(0, c["max_pos"], (t,), generator=g, device=DEVICE)
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEVICE)
                          / c["rot"])
        ang = torch.arange(c["max_pos"], dtype=torch.float64, device=DEVICE)[:, None] * inv
        s.cs = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s.q_out = torch.empty((t, hq, d), dtype=dt, device=DEVICE)
        if own:
            pkv = _pkv()
            code = {"f16": pkv.PKV_F16, "bf16": pkv.PKV_BF16, "e4m3": pkv.PKV_FP8_E4M3,
                    "e4m3tok": pkv.PKV_FP8_E4M3_TOKEN}[c["cache"]]
            s.desc = pkv.make_desc(blocks, PAGE, hkv, hq, d, code, s.ks, s.vs)
        return s
    b = c["batch"]
    order = torch.randperm(b, generator=g, device=DEVICE).tolist()
    if c["op"] == "shared":
        shared = c["prefix"] // PAGE
        spread = _spread(c["lo"], c["hi"], b)
        lens = [c["prefix"] + spread[i] for i in order]
        own_pages = [-(-(n - c["prefix"]) // PAGE) for n in lens]
    else:
        shared = 0
        if c["op"] == "decode":
            spread = _spread(c["lo"], c["hi"], b)
            lens = [spread[i] for i in order]
        else:
            chunks = _spread(c["chunk_lo"], c["chunk_hi"], b)
            pasts = _spread(c["past_lo"], c["past_hi"], b)
            s.chunks = [chunks[i] for i in order]
            lens = [chunks[i] + pasts[i] for i in order]
        own_pages = [-(-n // PAGE) for n in lens]
    mbs = shared + max(own_pages)
    blocks = shared + sum(own_pages) + 3
    _pool(s, c, blocks, g)
    perm = torch.randperm(blocks, generator=g, device=DEVICE).to(torch.int32)
    s.tables = torch.zeros((b, mbs), dtype=torch.int32, device=DEVICE)
    s.tables[:, :shared] = perm[:shared]
    at = shared
    for i, n in enumerate(own_pages):
        s.tables[i, shared:shared + n] = perm[at:at + n]
        at += n
    s.prefix = perm[:shared].contiguous()
    s.lens_host = lens
    s.lens = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    rows = b
    if c["op"] == "prefill":
        starts = [0]
        for n in s.chunks:
            starts.append(starts[-1] + n)
        s.starts_host = starts
        s.starts = torch.tensor(starts, dtype=torch.int32, device=DEVICE)
        rows = starts[-1]
        n = torch.tensor(s.chunks, device=DEVICE)
        s.row_seq = torch.repeat_interleave(torch.arange(b, device=DEVICE), n)  # of a row: its
        s.row_at = torch.arange(rows, device=DEVICE) - s.starts[s.row_seq]      # place there
    # scores of a spread that the cap bends
    gain = 6.0 if c.get("cap") else 1.0
    s.q = (gain * torch.randn((rows, hq, d), generator=g, device=DEVICE)).to(dt)
    s.slopes = _alibi(hq) if c.get("alibi") else None
    if own:
        pkv = _pkv()
        code = {"f16": pkv.PKV_F16, "bf16": pkv.PKV_BF16, "e4m3": pkv.PKV_FP8_E4M3,
                "e4m3tok": pkv.PKV_FP8_E4M3_TOKEN}[c["cache"]]
        s.desc = pkv.make_desc(blocks, PAGE, hkv, hq, d, code, s.ks, s.vs)
        s.out = torch.empty_like(s.q)
        if c["op"] == "shared":
            n = pkv.pkv_shared_prefix_workspace_bytes(s.desc, b, shared, mbs)
        else:
            n = pkv.pkv_decode_workspace_bytes(s.desc, b, mbs)
        s.ws = torch.zeros(n, dtype=torch.uint8, device=DEVICE)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    s, c = state, state.c
    if own:
        pkv = _pkv()
        if c["op"] == "append":
            pkv.pkv_kv_append_rope(s.desc, s.kc, s.vc, s.slots, s.pos, s.cs, s.q, s.k, s.v,
                                   s.q_out, interleaved=c["interleaved"])
            return _append_outputs(s)
        if c["op"] == "shared":
            pkv.pkv_paged_decode_attention_shared_prefix(
                s.desc, s.q, s.kc, s.vc, s.prefix, s.tables, s.lens, s.scale, s.out, s.ws)
        elif c["op"] == "decode":
            pkv.pkv_paged_decode_attention_biased(
                s.desc, s.q, s.kc, s.vc, s.tables, s.lens, s.scale, s.out, s.ws,
                softcap=c["cap"], alibi_slopes=s.slopes, window=c["window"])
        else:
            pkv.pkv_paged_prefill_attention_biased(
                s.desc, s.q, s.kc, s.vc, s.tables, s.lens, s.starts, max(s.chunks), s.scale,
                s.out, softcap=c["cap"], alibi_slopes=s.slopes)
        return s.out
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "shared":
        return _plain_shared(s)
    if c["op"] == "decode":
        return _plain_decode(s)
    return _plain_prefill(s)


def _append_outputs(s):
    out = {"q": s.q_out, "k_cache": s.kc, "v_cache": s.vc}
    if s.c["cache"] == "e4m3tok":
        out["scales"] = s.ks
    return out


def _rotate(x, cos, sin, rot, interleaved):
    """x [t][heads][d] in 32 bits; cos, sin [t][rot / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    return y


def _plain_append(s):
    c = s.c
    cs = s.cs[s.pos]
    cos, sin = cs[:, :c["rot"] // 2], cs[:, c["rot"] // 2:]
    s.q_out.copy_(_rotate(s.q.float(), cos, sin, c["rot"], c["interleaved"]))
    k = _rotate(s.k.float(), cos, sin, c["rot"], c["interleaved"])
    v = s.v.float()
    blk, off = s.slots // PAGE, s.slots % PAGE
    if c["cache"] == "e4m3":
        k, v = k / s.ks[None, :, None], v / s.vs[None, :, None]
    elif c["cache"] == "e4m3tok":
        top = torch.stack([k, v], 2).abs().amax(-1)
        top = torch.where(top > 0, top / 448.0, torch.ones_like(top))
        s.ks[blk, :, :, off] = top
        k, v = k / top[:, :, 0, None], v / top[:, :, 1, None]
    _store(s.kc, blk, off, k)
    _store(s.vc, blk, off, v)
    return _append_outputs(s)


def _store(cache, blk, off, x):
    if cache.dtype == torch.float8_e4m3fn:
        x = x.clamp(-448, 448).to(cache.dtype)
        cache.view(torch.uint8)[blk, :, off] = x.view(torch.uint8)
    else:
        cache[blk, :, off] = x.to(cache.dtype)


def _rows(s, ids, which, dtype):
    """Cache rows of the blocks ids [...][pages]: [...][pages * 16][kv_heads][d]."""
    cache = s.kc if which == 0 else s.vc
    ids = ids.long()
    if s.c["cache"].startswith("e4m3"):
        x = cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).to(dtype)
        if s.c["cache"] == "e4m3":
            x = x * (s.ks if which == 0 else s.vs).to(dtype)[:, None, None]
        else:
            x = x * s.ks[ids][..., which, :].to(dtype)[..., None]
    else:
        x = cache[ids].to(dtype)
    x = x.transpose(-3, -2)
    return x.reshape(*ids.shape[:-1], ids.shape[-1] * PAGE, s.c["kv_heads"], s.c["d"])


def _bias(s, x, u, t, slopes):
    """The cap and the distance bias; u - t broadcasts against x [heads...]."""
    c = s.c
    if c.get("cap"):
        x = c["cap"] * torch.tanh(x / c["cap"])
    if slopes is not None:
        x = x + slopes * (u - t)
    return x


def _softmax_dot(x, see, v, eq):
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    den = p.sum(-1, keepdim=True)
    return torch.einsum(eq, p / torch.where(den > 0, den, torch.ones_like(den)), v)


def _plain_shared(s):
    c = s.c
    hkv, d, b = c["kv_heads"], c["d"], c["batch"]
    grp = c["q_heads"] // hkv
    q = s.q.float().view(b, hkv, grp, d) * s.scale
    kp, vp = _rows(s, s.prefix, 0, torch.float32), _rows(s, s.prefix, 1, torch.float32)
    shared = c["prefix"] // PAGE
    ko = _rows(s, s.tables[:, shared:], 0, torch.float32)
    vo = _rows(s, s.tables[:, shared:], 1, torch.float32)
    u = torch.arange(ko.shape[1], device=DEVICE)
    see = u[None, :] < (s.lens - c["prefix"])[:, None]
    xp = torch.einsum("bhgd,nhd->bhgn", q, kp)
    xo = torch.einsum("bhgd,bnhd->bhgn", q, ko)
    xo = xo.masked_fill(~see[:, None, None], -math.inf)
    m = torch.maximum(xp.amax(-1, keepdim=True), xo.amax(-1, keepdim=True))
    pp, po = torch.exp(xp - m), torch.exp(xo - m)
    o = torch.einsum("bhgn,nhd->bhgd", pp, vp) + torch.einsum("bhgn,bnhd->bhgd", po, vo)
    o = o / (pp.sum(-1, keepdim=True) + po.sum(-1, keepdim=True))
    return o.reshape(b, c["q_heads"], d).to(s.dt)


def _plain_decode(s):
    c = s.c
    hkv, d, b = c["kv_heads"], c["d"], c["batch"]
    grp = c["q_heads"] // hkv
    q = s.q.float().view(b, hkv, grp, d) * s.scale
    k, v = _rows(s, s.tables, 0, torch.float32), _rows(s, s.tables, 1, torch.float32)
    u = torch.arange(k.shape[1], device=DEVICE)
    t = s.lens[:, None].long() - 1
    see = u[None, :] <= t
    if c["window"]:
        see = see & (u[None, :] > t - c["window"])
    slopes = None if s.slopes is None else s.slopes.view(1, hkv, grp, 1)
    x = torch.einsum("bhgd,bnhd->bhgn", q, k)
    x = _bias(s, x, u[None, None, None], t[:, None, None].float(), slopes)
    o = _softmax_dot(x, see[:, None, None], v, "bhgn,bnhd->bhgd")
    return o.reshape(b, c["q_heads"], d).to(s.dt)


def _plain_prefill(s):
    c = s.c
    hkv, d = c["kv_heads"], c["d"]
    grp = c["q_heads"] // hkv
    most = max(s.chunks)
    q = torch.zeros((c["batch"], most, c["q_heads"], d), device=DEVICE)
    q[s.row_seq, s.row_at] = s.q.float() * s.scale  # padded to the longest chunk
    q = q.view(c["batch"], most, hkv, grp, d)
    k, v = _rows(s, s.tables, 0, torch.float32), _rows(s, s.tables, 1, torch.float32)
    u = torch.arange(k.shape[1], device=DEVICE)
    first = s.lens - (s.starts[1:] - s.starts[:-1])  # position of a chunk's row 0
    t = (first[:, None] + torch.arange(most, device=DEVICE))[:, None, None, :, None]
    slopes = None if s.slopes is None else s.slopes.view(hkv, grp, 1, 1)
    x = torch.einsum("brhgd,bnhd->bhgrn", q, k)
    x = _bias(s, x, u.float(), t.float(), slopes)
    o = _softmax_dot(x, u <= t, v, "bhgrn,bnhd->brhgd")
    return o.reshape(c["batch"], most, c["q_heads"], d)[s.row_seq, s.row_at].to(s.dt)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions in 64 bits, one sequence and KV head at a time."""
    s = prepare(case, seed)
    c = s.c
    f8 = torch.float64
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["d"]
    grp = hq // hkv
    if c["op"] == "append":
        rot = c["rot"]
        half = rot // 2
        ang = s.cs.to(f8)[s.pos]
        z = torch.complex(ang[:, :half], ang[:, half:])[:, None]  # cos + i sin

        def turn(x):
            x = x.to(f8)
            if c["interleaved"]:
                w = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], half, 2)
                                          .contiguous()) * z
                w = torch.view_as_real(w).reshape(*x.shape[:-1], rot)
            else:
                w = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous()) * z
                w = torch.cat([w.real, w.imag], -1)
            return torch.cat([w, x[..., rot:]], -1)

        q, new = turn(s.q), [turn(s.k), s.v.to(f8)]
        blk = torch.div(s.slots, PAGE, rounding_mode="floor")
        off = s.slots - blk * PAGE
        out = {"q": q}
        scales = None if c["cache"] != "e4m3tok" else s.ks.to(f8)
        for i, (name, cache) in enumerate((("k_cache", s.kc), ("v_cache", s.vc))):
            x, full = new[i], cache.to(f8)
            if c["cache"] == "e4m3":
                x = x / (s.ks if i == 0 else s.vs).to(f8)[None, :, None]
            elif scales is not None:
                top = x.abs().amax(-1) / 448.0
                scales[blk, :, i, off] = top
                x = x / top[..., None]
            full[blk, :, off] = x.clamp(-448.0, 448.0) if c["cache"].startswith("e4m3") else x
            out[name] = full
        if scales is not None:
            out["scales"] = scales
        return out
    out = torch.zeros(s.q.shape, dtype=f8, device=DEVICE)
    shared = c["prefix"] // PAGE if c["op"] == "shared" else 0
    for b, ln in enumerate(s.lens_host):
        pages = -(-ln // PAGE)
        if c["op"] == "shared":
            ids = torch.cat([s.prefix, s.tables[b, shared:pages]])
        else:
            ids = s.tables[b, :pages]
        k, v = _exact_rows(s, ids, ln)
        n = s.chunks[b] if c["op"] == "prefill" else 1
        first = s.starts_host[b] if c["op"] == "prefill" else b
        t = torch.arange(ln - n, ln, device=DEVICE, dtype=f8)[:, None]
        u = torch.arange(ln, device=DEVICE, dtype=f8)[None]
        hidden = u > t
        if c.get("window"):
            hidden = hidden | (u <= t - c["window"])
        for h in range(hq):
            x = (s.q[first:first + n, h].to(f8) @ k[h // grp].T) * s.scale
            if c.get("cap"):
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if s.slopes is not None:
                x = x - s.slopes[h].to(f8) * (t - u)
            x[hidden] = -math.inf
            out[first:first + n, h] = torch.softmax(x, -1) @ v[h // grp]
    return out


def _exact_rows(s, ids, n):
    """K and V of one sequence, [kv_heads][n][d], in 64 bits."""
    pair = []
    for i, cache in enumerate((s.kc, s.vc)):
        x = cache.view(torch.uint8)[ids.long()].view(cache.dtype) if cache.element_size() == 1 \
            else cache[ids.long()]
        x = x.double()
        if s.c["cache"] == "e4m3":
            x *= (s.ks, s.vs)[i].double()[None, :, None, None]
        elif s.c["cache"] == "e4m3tok":
            x *= s.ks[ids.long(), :, i].double()[..., None]
        pair.append(x.permute(1, 0, 2, 3).flatten(1, 2)[:, :n])
    return pair
