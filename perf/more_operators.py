"""Workloads of the cache's speculative and eviction operators: attention for a
tree of drafted tokens and the acceptance of a path through it, decode attention
that accumulates each cached row's attention weight, and the eviction that goes
by those weights.

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
_BYTES = {"f16": 2, "bf16": 2, "e4m3": 1, "e4m3tok": 1}


def _pkv():
    import paged_kv_cache_250_gb300 as pkv
    return pkv


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a chat with one user, a small draft behind a short context: latency counts
        {"name": "tree_1", "op": "tree", "batch": 1, "q_heads": 32, "kv_heads": 8, "d": 128,
         "cache": "bf16", "past_lo": 701, "past_hi": 701, "nodes_lo": 7, "nodes_hi": 7},
        # a serving batch of ragged contexts, trees of every size up to the largest
        {"name": "tree_batch", "op": "tree", "batch": 32, "q_heads": 32, "kv_heads": 8, "d": 128,
         "cache": "bf16", "past_lo": 1, "past_hi": 4096, "nodes_lo": 1, "nodes_hi": 64},
        # eight query heads per KV head, long contexts, whole trees
        {"name": "tree_long", "op": "tree", "batch": 8, "q_heads": 64, "kv_heads": 8, "d": 128,
         "cache": "bf16", "past_lo": 32704, "past_hi": 32704, "nodes_lo": 64, "nodes_hi": 64},
        # the step after tree_1: a few rows of one sequence move up
        {"name": "accept_1", "op": "accept", "batch": 1, "kv_heads": 8, "group": 4, "d": 128,
         "cache": "bf16", "past_lo": 701, "past_hi": 701, "nodes_lo": 7, "nodes_hi": 7,
         "path": 3},
        # a large batch with whole trees in a cache of one scale per row
        {"name": "accept_batch_e4m3tok", "op": "accept", "batch": 256, "kv_heads": 8, "group": 4,
         "d": 128, "cache": "e4m3tok", "past_lo": 1, "past_hi": 4096, "nodes_lo": 16,
         "nodes_hi": 64, "path": 12},
        # one sequence, one KV head per query head, odd length
        {"name": "scored_1", "op": "scored", "batch": 1, "q_heads": 32, "kv_heads": 32, "d": 128,
         "cache": "f16", "lo": 701, "hi": 701, "decay": 1.0},
        # a serving batch of ragged lengths
        {"name": "scored_batch", "op": "scored", "batch": 32, "q_heads": 32, "kv_heads": 8,
         "d": 128, "cache": "bf16", "lo": 1, "hi": 4096, "decay": 1.0},
        # a large batch in a cache of one scale per row, older steps forgotten by and by
        {"name": "scored_long_e4m3tok", "op": "scored", "batch": 64, "q_heads": 32, "kv_heads": 8,
         "d": 128, "cache": "e4m3tok", "lo": 8192, "hi": 8192, "decay": 0.98},
        # a full cache that lets one row go at every step
        {"name": "evict_step", "op": "evict", "batch": 32, "kv_heads": 8, "group": 4, "d": 128,
         "cache": "bf16", "lo": 2049, "hi": 2049, "budget": 2048, "fresh": 1, "sinks": 4,
         "recent": 512},
        # the same every 128 steps, a larger batch in an E4M3 cache
        {"name": "evict_period_e4m3", "op": "evict", "batch": 64, "kv_heads": 8, "group": 4,
         "d": 128, "cache": "e4m3", "lo": 4224, "hi": 4224, "budget": 4096, "fresh": 128,
         "sinks": 4, "recent": 1024},
        # long prompts cut down before the first decode step, ragged
        {"name": "evict_prompts", "op": "evict", "batch": 8, "kv_heads": 8, "group": 8, "d": 128,
         "cache": "bf16", "lo": 3000, "hi": 32768, "budget": 4096, "fresh": 0, "sinks": 16,
         "recent": 512},
        # one very long prompt
        {"name": "evict_prompt_1_e4m3tok", "op": "evict", "batch": 1, "kv_heads": 8, "group": 4,
         "d": 128, "cache": "e4m3tok", "lo": 131072, "hi": 131072, "budget": 8192, "fresh": 0,
         "sinks": 4, "recent": 1024},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "accept", "scored", "scored", "evict", "evict"])
    g = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128, 128])
    cache = rng.choice(["f16", "bf16"] if op == "tree" else ["f16", "bf16", "e4m3", "e4m3tok"])
    d = 128 if cache.startswith("e4m3") else d
    if op in ("tree", "accept"):
        most = _log_int(rng, 1, 64)
        c = {"op": op, "batch": _log_int(rng, 1, 64), "kv_heads": hkv, "d": d, "cache": cache,
             "nodes_lo": _log_int(rng, 1, most), "nodes_hi": most}
        past = _log_int(rng, 1, 32705) - 1
        if op == "tree":
            past = min(past, (8 * 64 * 64 * 32704) // (c["batch"] * g * hkv * most))
            return {**c, "q_heads": g * hkv, "past_lo": past // rng.choice([1, 2, 8]),
                    "past_hi": past}
        past = min(past, 8192)
        return {**c, "group": g, "past_lo": past // 2, "past_hi": past,
                "path": rng.randint(0, min(most, 16))}
    if op == "scored":
        hi = _log_int(rng, 1, 16384)
        return {"op": op, "batch": _log_int(rng, 1, 32), "q_heads": g * hkv, "kv_heads": hkv,
                "d": d, "cache": cache, "lo": _log_int(rng, 1, hi), "hi": hi,
                "decay": rng.choice([1.0, 1.0, 0.9, 0.0])}
    budget = _log_int(rng, 1, 8192)
    sinks = min(budget // 4, rng.choice([0, 4, 17]))
    recent = rng.randint(0, budget - sinks)
    fresh = rng.choice([0, 1, _log_int(rng, 1, 256)])
    if fresh:  # a cache that was full before the last `fresh` tokens came
        recent = max(recent, min(fresh, budget - sinks))
        hi = lo = budget + fresh
    else:
        hi = _log_int(rng, 1, 32768)
        lo = _log_int(rng, 1, hi)
    return {"op": op, "batch": _log_int(rng, 1, 32), "kv_heads": hkv, "group": g, "d": d,
            "cache": cache, "lo": lo, "hi": hi, "budget": budget, "fresh": fresh, "sinks": sinks,
            "recent": recent}


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], the same for every seed."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _row_bytes(c):
    """Bytes of a cached token of one KV head: K, V and their scales."""
    return 2 * c["d"] * _BYTES[c["cache"]] + (8 if c["cache"] == "e4m3tok" else 0)


def work(case):
    c = case
    b, hkv = c["batch"], c["kv_heads"]
    if c["op"] in ("tree", "accept"):
        pasts = _spread(c["past_lo"], c["past_hi"], b)
        nodes = _spread(c["nodes_lo"], c["nodes_hi"], b)
    if c["op"] == "tree":
        # a node sees the past and itself (its ancestors come on top)
        seen = sum(n * (p + 1) for n, p in zip(nodes, pasts))
        rows = sum(nodes)
        toks = rows + sum(pasts)
        return {"bytes": toks * hkv * _row_bytes(c) + rows * (c["q_heads"] * c["d"] * 4 + 8)
                + toks // PAGE * 4 + 8 * b, "flops": 4 * c["d"] * c["q_heads"] * seen}
    if c["op"] == "accept":
        moved = sum(min(c["path"], n) for n in nodes)
        return {"bytes": 2 * moved * hkv * _row_bytes(c) + 4 * moved + 16 * b, "flops": 0}
    lens = _spread(c["lo"], c["hi"], b)
    if c["op"] == "scored":
        toks = sum(lens)
        return {"bytes": toks * hkv * (_row_bytes(c) + 8) + b * c["q_heads"] * c["d"] * 4
                + toks // PAGE * 4 + 4 * b,
                "flops": (4 * c["d"] + 2) * c["q_heads"] * toks}
    # eviction: every row's weight and position, and the rows that change places
    read = moved = 0
    for n in lens:
        if n <= c["budget"]:
            read += 4 * (c["fresh"] if c["fresh"] else n)  # the new rows' positions
            continue
        read += 4 * n + (4 * c["budget"] if c["fresh"] else 4 * c["budget"])
        free = c["budget"] - c["sinks"] - c["recent"]
        if c["fresh"]:
            moved += min(c["fresh"], c["recent"])
        else:
            last = min(c["recent"], n - c["budget"])
            others = n - c["sinks"] - c["recent"]
            moved += last + free * max(0, n - c["budget"] - c["recent"]) // max(1, others)
    return {"bytes": hkv * (read + moved * (2 * _row_bytes(c) + 16)) + 20 * b, "flops": 0}


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


def prepare(case, seed):
    c = dict(case)
    c.setdefault("q_heads", c["kv_heads"] * c.get("group", 1))
    g = torch.Generator(device=DEVICE).manual_seed(1_000_003 * (int(seed) % 1_000_003) + 29)
    gc = torch.Generator().manual_seed(1_000_003 * (int(seed) % 1_000_003) + 31)
    s = State()
    s.c = c
    b, hq, hkv, d = c["batch"], c["q_heads"], c["kv_heads"], c["d"]
    s.dt = _DT.get(c["cache"], torch.bfloat16)
    s.scale = 1.0 / math.sqrt(d)
    order = torch.randperm(b, generator=gc).tolist()
    if c["op"] in ("tree", "accept"):
        pasts = _spread(c["past_lo"], c["past_hi"], b)
        nodes = _spread(c["nodes_lo"], c["nodes_hi"], b)
        # long contexts with any tree, the same pairs for every seed
        mixed = torch.randperm(b, generator=torch.Generator().manual_seed(7)).tolist()
        s.nodes = [nodes[mixed[i]] for i in order]
        lens = [pasts[i] + n for i, n in zip(order, s.nodes)]
    else:
        spread = _spread(c["lo"], c["hi"], b)
        lens = [spread[i] for i in order]
    s.lens_host = lens
    s.lens = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    # whole tables, short ones filled up with a block that nobody owns
    pages = torch.tensor([-(-n // PAGE) for n in lens])
    mbs, total = max(1, int(pages.max())), int(pages.sum())
    blocks = total + 3
    _pool(s, c, blocks, g)
    perm = torch.randperm(blocks, generator=gc).to(torch.int32)
    tables = torch.full((b, mbs), int(perm[total]), dtype=torch.int32)
    tables[torch.arange(mbs)[None, :] < pages[:, None]] = perm[:total]
    s.tables = tables.to(DEVICE)
    if c["op"] in ("tree", "accept"):
        starts = [0]
        for n in s.nodes:
            starts.append(starts[-1] + n)
        s.starts_host = starts
        s.starts = torch.tensor(starts, dtype=torch.int32, device=DEVICE)
        # a node hangs on one of those before it: a row's word has its ancestors' bits
        # and its own
        most = max(s.nodes)
        words = torch.zeros((b, most), dtype=torch.int64)
        for j in range(most):
            bit = 1 << j if j < 63 else -(1 << 63)
            words[:, j] = bit
            if j > 0:
                up = (torch.rand(b, generator=gc) * j).long()
                words[:, j] |= words[torch.arange(b), up]
        real = torch.arange(most)[None, :] < torch.tensor(s.nodes)[:, None]
        s.mask = words[real].to(DEVICE)
        n = torch.tensor(s.nodes, device=DEVICE)
        s.row_seq = torch.repeat_interleave(torch.arange(b, device=DEVICE), n)
        s.row_at = torch.arange(starts[-1], device=DEVICE) - s.starts[s.row_seq]
        if c["op"] == "tree":
            s.q = torch.randn((starts[-1], hq, d), generator=g, device=DEVICE).to(s.dt)
        else:  # nodes in rising order, as many as the tree has
            steps = c["path"]
            pick = torch.rand((b, most), generator=gc).masked_fill(~real, 2.0).argsort(1)
            s.path_host = [sorted(pick[i, :min(steps, k)].tolist())
                           for i, k in enumerate(s.nodes)]
            path = torch.zeros((b, max(1, steps)), dtype=torch.int32)
            for i, p in enumerate(s.path_host):
                path[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
            s.path = path.to(DEVICE)
            s.path_lens = torch.tensor([len(p) for p in s.path_host], dtype=torch.int32,
                                       device=DEVICE)
            s.new_lens = torch.empty_like(s.lens)
    else:
        # weights summed over many steps: few rows have most of them, some none
        w = torch.exp(2.0 * torch.randn((blocks, hkv, PAGE), generator=g, device=DEVICE))
        w[torch.rand(w.shape, generator=g, device=DEVICE) < 0.05] = 0.0
        s.weights = w
    if c["op"] == "scored":
        s.q = torch.randn((b, hq, d), generator=g, device=DEVICE).to(s.dt)
    if c["op"] == "evict":
        s.new_lens = torch.empty_like(s.lens)
        s.positions = torch.zeros((blocks, hkv, PAGE), dtype=torch.int32, device=DEVICE)
        if c["fresh"]:
            # a cache of `budget` rows that lost others before: any order, the sinks in it
            kept = c["budget"]
            s.old_lens = torch.full_like(s.lens, kept)
            s.num_tokens = s.lens * 3
            before = 3 * c["hi"] - c["fresh"]
            far = torch.rand((b, hkv, before), generator=g, device=DEVICE)
            far[:, :, :c["sinks"]] = -1.0
            pos = far.argsort(-1)[:, :, :kept]
            pos = pos.gather(2, torch.rand((b, hkv, kept), generator=g, device=DEVICE).argsort(-1))
            whole = torch.zeros((b, hkv, mbs * PAGE), dtype=torch.int32, device=DEVICE)
            whole[:, :, :kept] = pos
            s.positions[s.tables.long()] = whole.view(b, hkv, mbs, PAGE).transpose(1, 2)
        else:
            s.old_lens = torch.zeros_like(s.lens)
            s.num_tokens = s.lens.clone()
            s.scored = s.weights.clone()
    if own:
        pkv = _pkv()
        code = {"f16": pkv.PKV_F16, "bf16": pkv.PKV_BF16, "e4m3": pkv.PKV_FP8_E4M3,
                "e4m3tok": pkv.PKV_FP8_E4M3_TOKEN}[c["cache"]]
        s.desc = pkv.make_desc(blocks, PAGE, hkv, hq, d, code, s.ks, s.vs)
        if c["op"] == "tree":
            s.out = torch.empty_like(s.q)
            n = pkv.pkv_tree_workspace_bytes(s.desc, b, max(s.nodes), mbs)
            s.ws = torch.zeros(n, dtype=torch.uint8, device=DEVICE)
        elif c["op"] == "scored":
            s.out = torch.empty_like(s.q)
            n = pkv.pkv_scored_workspace_bytes(s.desc, b, mbs)
            s.ws = torch.zeros(n, dtype=torch.uint8, device=DEVICE)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    s, c = state, state.c
    if c["op"] == "evict":
        if c["fresh"]:  # the tokens that came since the last pass
            s.num_tokens += c["fresh"]
        else:  # the weights of another prompt's rows
            s.weights.copy_(s.scored)
    if own:
        pkv = _pkv()
        if c["op"] == "tree":
            pkv.pkv_paged_tree_attention(s.desc, s.q, s.kc, s.vc, s.tables, s.lens, s.starts,
                                         max(s.nodes), s.mask, s.scale, s.out, s.ws)
            return s.out
        if c["op"] == "accept":
            pkv.pkv_kv_accept_path(s.desc, s.kc, s.vc, s.tables, s.lens, s.starts, s.path,
                                   s.path_lens, s.new_lens)
            return _cache_outputs(s)
        if c["op"] == "scored":
            pkv.pkv_paged_decode_attention_scored(s.desc, s.q, s.kc, s.vc, s.tables, s.lens,
                                                  s.weights, s.scale, s.out, s.ws,
                                                  decay=c["decay"])
            return {"out": s.out, "weights": s.weights}
        pkv.pkv_kv_evict(s.desc, s.kc, s.vc, s.weights, s.positions, s.tables, s.lens, s.old_lens,
                         s.num_tokens, c["budget"], c["sinks"], c["recent"], s.new_lens)
        return _cache_outputs(s)
    if c["op"] == "tree":
        return _plain_tree(s)
    if c["op"] == "accept":
        return _plain_accept(s)
    if c["op"] == "scored":
        return _plain_scored(s)
    return _plain_evict(s)


def _cache_outputs(s):
    out = {"k_cache": s.kc, "v_cache": s.vc, "new_lens": s.new_lens}
    if s.c["cache"] == "e4m3tok":
        out["scales"] = s.ks
    if s.c["op"] == "evict":
        out["weights"], out["positions"] = s.weights, s.positions
    return out


def _rows(s, which):
    """Cache rows of all sequences: [batch][table's tokens][kv_heads][d], in 32 bits."""
    cache = s.kc if which == 0 else s.vc
    ids = s.tables.long()
    if s.c["cache"].startswith("e4m3"):
        x = cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
        if s.c["cache"] == "e4m3":
            x = x * (s.ks if which == 0 else s.vs)[:, None, None]
        else:
            x = x * s.ks[ids][..., which, :, None]
    else:
        x = cache[ids].float()
    x = x.transpose(2, 3)
    return x.reshape(ids.shape[0], ids.shape[1] * PAGE, s.c["kv_heads"], s.c["d"])


def _softmax(x, see):
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    den = p.sum(-1, keepdim=True)
    return p / torch.where(den > 0, den, torch.ones_like(den))


def _plain_tree(s):
    c = s.c
    b, hkv, d = c["batch"], c["kv_heads"], c["d"]
    grp = c["q_heads"] // hkv
    most = max(s.nodes)
    q = torch.zeros((b, most, c["q_heads"], d), device=DEVICE)
    q[s.row_seq, s.row_at] = s.q.float() * s.scale  # padded to the largest tree
    words = torch.zeros((b, most), dtype=torch.int64, device=DEVICE)
    words[s.row_seq, s.row_at] = s.mask
    k, v = _rows(s, 0), _rows(s, 1)
    u = torch.arange(k.shape[1], device=DEVICE)
    first = s.lens - (s.starts[1:] - s.starts[:-1])  # position of a tree's node 0
    node = u[None, :] - first[:, None]
    bits = (words[:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1
    see = (node < 0)[:, None, :] | ((u[None, :] < s.lens[:, None])[:, None, :] & (bits == 1))
    x = torch.einsum("brhgd,bnhd->bhgrn", q.view(b, most, hkv, grp, d), k)
    o = torch.einsum("bhgrn,bnhd->brhgd", _softmax(x, see[:, None, None]), v)
    return o.reshape(b, most, c["q_heads"], d)[s.row_seq, s.row_at].to(s.dt)


def _places(s, at):
    """Block and offset of the rows at [batch][...] of each sequence."""
    page = torch.div(at, PAGE, rounding_mode="floor")
    blk = s.tables.long().gather(1, page.reshape(at.shape[0], -1)).reshape(at.shape)
    return blk, at - page * PAGE


def _plain_accept(s):
    i = torch.arange(s.path.shape[1], device=DEVICE)[None, :]
    nodes = (s.starts[1:] - s.starts[:-1]).long()
    base = (s.lens - nodes)[:, None]
    # steps that a sequence's path does not have write a row to itself
    still = torch.minimum(i.expand(base.shape[0], -1), nodes[:, None] - 1)
    src = torch.where(i < s.path_lens[:, None], s.path.long(), still)
    dst = torch.where(i < s.path_lens[:, None], i, still)
    sb, so = _places(s, base + src)
    db, do = _places(s, base + dst)
    _copy(s.kc, (sb, slice(None), so), (db, slice(None), do))
    _copy(s.vc, (sb, slice(None), so), (db, slice(None), do))
    if s.c["cache"] == "e4m3tok":
        _copy(s.ks, (sb, slice(None), slice(None), so), (db, slice(None), slice(None), do))
    s.new_lens.copy_(base[:, 0] + s.path_lens)
    return _cache_outputs(s)


def _copy(pool, src, dst):
    pool = pool.view(torch.uint8) if pool.element_size() == 1 else pool
    pool[dst] = pool[src]


def _plain_scored(s):
    c = s.c
    b, hkv, d = c["batch"], c["kv_heads"], c["d"]
    grp = c["q_heads"] // hkv
    q = s.q.float().view(b, hkv, grp, d) * s.scale
    k, v = _rows(s, 0), _rows(s, 1)
    n = k.shape[1]
    u = torch.arange(n, device=DEVICE)
    see = (u[None, :] < s.lens[:, None])[:, None, None]
    p = _softmax(torch.einsum("bhgd,bnhd->bhgn", q, k), see)
    o = torch.einsum("bhgn,bnhd->bhgd", p, v)
    ids = s.tables.long()
    old = s.weights[ids].transpose(1, 2).reshape(b, hkv, n)
    newest = (u[None, :] == s.lens[:, None] - 1)[:, None]
    w = torch.where(newest, torch.zeros_like(old), c["decay"] * old) + p.sum(2)
    w = torch.where(see[:, :, 0], w, old)
    s.weights[ids] = w.view(b, hkv, -1, PAGE).transpose(1, 2)
    return {"out": o.reshape(b, c["q_heads"], d).to(s.dt), "weights": s.weights}


def _plain_evict(s):
    c = s.c
    b, hkv, budget = c["batch"], c["kv_heads"], c["budget"]
    ids = s.tables.long()
    n = ids.shape[1] * PAGE
    u = torch.arange(n, device=DEVICE)[None, None, :]
    length, old = s.lens[:, None, None], s.old_lens[:, None, None]
    told = s.num_tokens[:, None, None]
    flat = (b, hkv, n)
    pos = s.positions[ids].transpose(1, 2).reshape(flat)
    pos = torch.where((u >= old) & (u < length), (told - length + u).int(), pos)
    w = s.weights[ids].transpose(1, 2).reshape(flat)
    guarded = (pos < c["sinks"]) | (pos >= told - c["recent"])
    key = torch.where(guarded, math.inf, w).masked_fill(u >= length, -math.inf)
    best = torch.sort(key, stable=True, descending=True).indices[..., :budget]
    keep = torch.zeros(flat, dtype=torch.bool, device=DEVICE).scatter_(2, best, True)
    keep = torch.where(length > budget, keep, u < length) & (u < length)
    hole = ~keep & (u < budget) & (length > budget)
    late = keep & (u >= budget)
    # the i-th late row goes to the i-th hole; all others to themselves
    place = torch.zeros((b, hkv, n + 1), dtype=torch.int64, device=DEVICE)
    place.scatter_(2, torch.where(hole, hole.cumsum(-1) - 1, n), u.expand(flat))
    to = torch.where(late, place.gather(2, (late.cumsum(-1) - 1).clamp_min(0)), u)[..., budget:]
    src = u[..., budget:].expand(to.shape)
    head = torch.arange(hkv, device=DEVICE)[None, :, None]
    s.positions[ids] = pos.view(b, hkv, -1, PAGE).transpose(1, 2)
    if src.shape[2]:
        sb, so = _places(s, src)
        db, do = _places(s, to)
        _copy(s.kc, (sb, head, so), (db, head, do))
        _copy(s.vc, (sb, head, so), (db, head, do))
        _copy(s.weights, (sb, head, so), (db, head, do))
        _copy(s.positions, (sb, head, so), (db, head, do))
        if c["cache"] == "e4m3tok":
            _copy(s.ks, (sb, head, slice(None), so), (db, head, slice(None), do))
    s.new_lens.copy_(s.lens.clamp_max(budget))
    return _cache_outputs(s)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The attention calls' definitions in 64 bits, one sequence and KV head at a
    time; the two calls that move rows compute no numbers."""
    if case["op"] in ("accept", "evict"):
        return None
    s = prepare(case, seed)
    c = s.c
    f8 = torch.float64
    grp = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s.q.shape, dtype=f8, device=DEVICE)
    weights = s.weights.double() if c["op"] == "scored" else None
    for b, ln in enumerate(s.lens_host):
        ids = s.tables[b, :-(-ln // PAGE)].long()
        k, v = _exact_rows(s, ids, ln)
        n = s.nodes[b] if c["op"] == "tree" else 1
        first = s.starts_host[b] if c["op"] == "tree" else b
        hidden = torch.zeros((n, ln), dtype=torch.bool, device=DEVICE)
        if c["op"] == "tree":
            i = torch.arange(n, device=DEVICE)
            hidden[:, ln - n:] = ((s.mask[first:first + n, None] >> i[None, :]) & 1) == 0
        at = torch.arange(ln, device=DEVICE)
        for h in range(c["kv_heads"]):
            mine = slice(h * grp, (h + 1) * grp)
            x = torch.einsum("rgd,nd->rgn", s.q[first:first + n, mine].to(f8), k[h]) * s.scale
            p = torch.softmax(x.masked_fill(hidden[:, None], -math.inf), -1)
            out[first:first + n, mine] = p @ v[h]
            if weights is not None:
                blk, off = ids[at // PAGE], at % PAGE
                before = weights[blk, h, off] * c["decay"]
                before[ln - 1] = 0.0
                weights[blk, h, off] = before + p[0].sum(0)
    return out if weights is None else {"out": out, "weights": weights}


def _exact_rows(s, ids, n):
    """K and V of one sequence, [kv_heads][n][d], in 64 bits."""
    pair = []
    for i, cache in enumerate((s.kc, s.vc)):
        x = cache.view(torch.uint8)[ids].view(cache.dtype) if cache.element_size() == 1 \
            else cache[ids]
        x = x.double()
        if s.c["cache"] == "e4m3":
            x *= (s.ks, s.vs)[i].double()[None, :, None, None]
        elif s.c["cache"] == "e4m3tok":
            x *= s.ks[ids, :, i].double()[..., None]
        pair.append(x.permute(1, 0, 2, 3).flatten(1, 2)[:, :n])
    return pair
