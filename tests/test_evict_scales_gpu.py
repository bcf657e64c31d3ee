"""Eviction from E4M3 caches by clusters of more than one CTA: the scales of rows that
move go with them (whole pools, byte for byte)."""
import pytest

from test_evict_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["e4m3", "e4m3tok"])
@pytest.mark.parametrize("Hq,Hkv,n,budget,weights", [(1, 1, 70001, 5000, "exp"),
                                                     (6, 3, 20000, 10000, "few"),
                                                     (2, 2, 9001, 17, "all"),
                                                     (8, 8, 40000, 8192, "exp")])
def test_long_sequences(cache, Hq, Hkv, n, budget, weights):
    c = Case([n], [n // 3], [n + 500], Hq, Hkv, 128, cache, 31, weights)
    c.check(budget, min(4, budget - 1), budget // 8)
    assert c.p.err.item() == 0


@pytest.mark.parametrize("wider", [300, 600, 1100, 49133])
def test_wide_tables(wider):
    """Clusters of two, four, eight and sixteen CTAs, most of which have no row."""
    c = Case([300, 90], [40, 0], [700, 90], cache="e4m3tok", seed=33, wider=wider)
    c.check(128, 4, 16)
    assert c.p.err.item() == 0
