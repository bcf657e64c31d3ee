"""A prefix block outside the pool: reported, and its positions left out of every
row, whichever way the prefix is read (once for the batch, or per sequence)."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import PAGE, Paged, attend, check
from test_shared_prefix_gpu import shared, workspace
from test_shared_prefix_passes_gpu import own_pass

pytestmark = pytest.mark.gpu


def without(p, q, b, pages):
    """Sequence b's row over the positions that are not in `pages` of the prefix."""
    n = p.lens[b]
    u = torch.arange(n)
    keep = ~torch.isin(u // PAGE, torch.tensor(pages))
    K, V = p.K[b][keep], p.V[b][keep]
    return attend(q[b].double(), K, V, p.scale, len(K) - 1)


CASES = [  # prefix, lens, Hq, Hkv, d, cache, a pass of its own
    # one tile of rows: streams of every second 128-token block
    (1040, [0, 5, 16, 17, 1039, 1040, 1041, 1100, 128, 130, 40, 700], 8, 8, 128, "bf16", True),
    # two tiles of rows, the last block of 128 tokens not whole
    (1040, [1040 + 3 * i for i in range(40)], 32, 4, 128, "f16", True),
    (4128, [900, 4128, 4140, 4127, 3, 4200, 4129], 16, 8, 64, "bf16", True),
    # read for every sequence
    (128, [129, 0, 5, 16, 128, 127, 400], 8, 1, 128, "f16", False),
]


@pytest.mark.parametrize("pages", [[0], [1, 6], [7, 8, 9], list(range(8)), [64], list(range(300))])
@pytest.mark.parametrize("case", CASES)
def test_a_bad_block_is_left_out(case, pages):
    prefix, lens, Hq, Hkv, d, cache, passes = case
    p = Paged(lens, Hq, Hkv, d, cache, 111, prefix=prefix)
    assert own_pass(p) == passes
    pages = [x for x in pages if x < prefix // PAGE]
    for i, x in enumerate(pages):
        p.prefix_blocks[x] = (p.NB, -1, 2 ** 30, -2 ** 31, 2 ** 31 - 1)[i % 5]
    q = p.queries(len(lens), 112, 2.0)
    ws = workspace(p)
    o = shared(p, q, ws=ws)
    assert p.err.item() == (pkv.PKV_ERR_BOUNDS if pages else 0)
    rows = range(min(len(lens), 12))
    ref = [without(p, q, b, pages) for b in rows]
    check(o[:12], torch.stack([r[0] for r in ref]), torch.stack([r[1] for r in ref]), "f32",
          str(pages[:8]))
    assert torch.equal(o, shared(p, q, ws=ws))


@pytest.mark.parametrize("longest", [1, 16, 17, 100, 128, 1030])
@pytest.mark.parametrize("prefix,Hq,Hkv,d,B,passes", [(1040, 8, 8, 128, 12, True),
                                                      (1040, 32, 4, 128, 40, True),
                                                      (1040, 8, 1, 64, 3, False)])
def test_blocks_behind_every_length_are_not_looked_up(longest, prefix, Hq, Hkv, d, B, passes):
    p = Paged([longest - i % 2 for i in range(B)], Hq, Hkv, d, "bf16", 113, prefix=prefix)
    assert own_pass(p) == passes
    p.prefix_blocks[-(-longest // PAGE):] = -1
    q = p.queries(B, 114, 2.0)
    o = shared(p, q)
    assert p.err.item() == 0
    ref = [without(p, q, b, []) for b in range(3)]
    check(o[:3], torch.stack([r[0] for r in ref]), torch.stack([r[1] for r in ref]), "f32")
