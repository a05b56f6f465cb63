"""Attention over a cache in 8 bits whose keys and values are very large or very small: the range of bf16 is that of fp32,
and scores are moderate where the queries make up for the keys."""

import pytest

from tests.test_tree8_gpu import BF16, Made

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [-100, -60, 60, 76])
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes,Hq", [([1, 2, 1, 3], 4), ([5, 7, 4, 6], 8), ([40, 70, 33, 20], 8)], ids=["few", "some", "many"])
def test_keys_and_values_of_any_size(gpu, nodes, Hq, d, tree, size):
    m = Made(gpu, [300, 0, 5000, 64], nodes, Hq, 2, d, 32, 16, BF16, tree=tree, seed=6, spread=0.0)
    factor = 2.0 ** size
    m.ks.mul_(factor)
    m.k.mul_(factor)
    m.q.mul_(1.0 / factor)
    m.check()
    m.vs.mul_(factor)
    m.v.mul_(factor)
    m.check()
