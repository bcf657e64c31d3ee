"""Sequences that the tree call cuts into every number of parts on both sides of
where the merge changes its ways (four and eight parts, 32 rows), held to the formula
in fp64."""
import pytest

from ops_harness import Paged, check
from test_tree_attention_gpu import expect, tree, trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 6, 8, 9, 10, 13])
@pytest.mark.parametrize("Hq,Hkv,nodes,d", [(4, 1, 7, 128), (8, 1, 4, 64), (2, 2, 33, 128),
                                            (8, 1, 16, 64), (8, 1, 17, 128), (8, 1, 64, 128)])
def test_parts(Hq, Hkv, nodes, d, blocks):
    for end in (0, 5):  # the last block full, or five tokens long
        ctx = 128 * blocks - (123 if end else 0)
        if ctx < nodes:
            continue
        p = Paged([ctx], Hq, Hkv, d, "bf16", 81 + blocks)
        q = p.queries(nodes, 82, 2.0)
        words = trees([nodes], 83)
        out = tree(p, q, [nodes], words)
        check(out, *expect(p, q, [nodes], words), "f32")
        assert p.err.item() == 0
