"""The bits of drafted trees: large ones, long chains, few words, bad parents; and the time that long chains take."""

import random

import numpy as np
import pytest
import torch

from io_aware_exact_04_gb300 import api
from test_serving_gpu import ints

pytestmark = pytest.mark.gpu


def plain(parents, nodes, words):
    """Row by row: a node's own bit and its parent's row; bits past the words left out."""
    out = np.zeros((len(parents), words), np.uint32)
    at = 0
    for n in nodes:
        for i in range(n):
            p = parents[at + i]
            if 0 <= p < i:
                out[at + i] = out[at + p]
            if i >> 5 < words:
                out[at + i, i >> 5] |= np.uint32(1 << (i & 31))
        at += n
    return torch.from_numpy(out.view(np.int32))


def draw(kind, nodes, seed):
    r = random.Random(seed)
    parents = []
    for n in nodes:
        for i in range(n):
            parents.append({"chain": i - 1, "forest": -1 if r.random() < 0.1 else r.randrange(i) if i else -1,
                            "near": i - 1 - r.randrange(min(i, 200)) if i else -9,
                            "bad": r.choice([i - 1, i, i + 3, -1, r.randrange(n), 1 << 30])}[kind])
    return parents


@pytest.mark.parametrize("kind", ["chain", "forest", "near", "bad"])
@pytest.mark.parametrize("nodes,words", [([1], 1), ([32, 0, 33, 1], 2), ([127, 128, 129], 5), ([7] * 300, 1), ([64] * 40, 7),
                                         ([1500, 3, 257], 47), ([300, 128, 5], 4), ([200, 700], 1), ([5000], 157)])
def test_masks(gpu, nodes, words, kind):
    parents = draw(kind, nodes, 1)
    T = sum(nodes)
    api.device_status(gpu)
    out = torch.full((T + 2, words), 0x5A5A5A5A, dtype=torch.int32, device=gpu)
    cu = ints([0] + np.cumsum(nodes).tolist(), gpu)
    # two rows that no sequence has stay as they are
    got = api.tree_mask(ints(parents + [0, 0], gpu), cu, words, out=out)
    torch.cuda.synchronize(gpu)
    assert torch.equal(got[:T].cpu(), plain(parents, nodes, words))
    assert (got[T:] == 0x5A5A5A5A).all()
    bad = max(nodes) > 32 * words or (kind == "bad" and any(p >= i for n, a in zip(nodes, np.cumsum([0] + nodes))
                                                            for i, p in enumerate(parents[a:a + n])))
    assert api.device_status(gpu)[0] == (6 if bad else 0)


def test_time_grows_with_the_nodes(gpu):
    """A chain of twice as many nodes (their bits past the first 32 left out, which is recorded) takes about twice
    as long: every node's walk to the root would make it four times."""
    def ms(n):
        parents, cu = torch.arange(-1, n - 1, dtype=torch.int32, device=gpu), ints([0, n], gpu)
        best = 1e9
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            got = api.tree_mask(parents, cu, 1)
            b.record()
            torch.cuda.synchronize(gpu)
            best = min(best, a.elapsed_time(b))
        assert got[31:].eq(-1).all()
        return best

    assert ms(40000) < 3 * ms(20000)
    assert api.device_status(gpu)[0] == 6
