"""Attention over a cache in 8 bits with scores of -inf alone: the definition's maximum is -inf, and the row is NaN, not
that of a node that sees nothing."""

import math

import pytest
import torch

from io_aware_exact_04_gb300 import api
from tests import serving_ref
from tests.test_tree8_gpu import BF16, FP16, Made

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("nodes,Hq", [([1, 2, 1, 3], 4), ([5, 7, 4, 6], 8), ([40, 70, 33, 20], 8)], ids=["few", "some", "many"])
@pytest.mark.parametrize("lens", [[300, 0, 1, 64], [0, 0, 0, 0], [20000, 5000, 0, 130]], ids=["short", "none", "long"])
def test_an_infinite_query_with_scores_of_minus_infinity(gpu, lens, nodes, Hq, dtype, d, tree):
    m = Made(gpu, lens, nodes, Hq, 2, d, 32, 16, dtype, tree=tree, tail=0, seed=6)
    m.k[:, :, 5] = -m.k[:, :, 5].abs() - 0.125
    x = m.kc.view(torch.uint8)
    x[..., 5] = torch.where(x[..., 5] == 0x7F, x[..., 5], (x[..., 5] & 0x7F).clamp(min=8) | 0x80)  # (0x7f: behind a length)
    want = m.check()
    at = serving_ref.offsets(m.nodes)
    hit = sorted({at[b] + i for b, n in enumerate(nodes) for i in (0, n // 2, n - 1)})
    head = 1
    m.q[hit, head, 5] = math.inf
    o, lse = m.call()
    assert api.device_status(gpu)[0] == 0
    expect = torch.zeros((m.T, Hq), dtype=torch.bool, device=gpu)
    for b, n in enumerate(nodes):
        for i in (0, n // 2, n - 1):
            expect[at[b] + i, head] = lens[b] > 0 or not tree or bool(m.per[b][i].any())
    assert torch.equal(o.isnan().all(-1), expect) and torch.equal(o.isnan().any(-1), expect)
    assert torch.equal(lse.isnan().t(), expect)
    assert torch.equal(o[~expect], want[0][~expect]) and torch.equal(lse.t()[~expect], want[1].t()[~expect])
