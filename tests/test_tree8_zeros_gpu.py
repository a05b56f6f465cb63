"""Attention over a cache in 8 bits with queries, keys and values of zero or nearly so: what a slot padded with zeros or
a warm-up call holds. A row whose scores are all equal gives the mean of the values that it sees, whatever factors the
kernels take out of rows and blocks without a value; scores that are masked stay masked.

FEW has few rows a sequence, MANY many: different kernels. MANY's numbers of nodes leave the second half of a tile of 64
empty, partly filled and full.
"""

import pytest
import torch

from tests import serving_ref
from tests.test_tree8_gpu import BF16, FP16, Made

pytestmark = pytest.mark.gpu
FEW = dict(lens=[300, 0, 33, 130], nodes=[1, 2, 1, 3], Hq=4, H=2)
MANY = dict(lens=[300, 0, 33, 130], nodes=[5, 20, 33, 40], Hq=16, H=2)
ALL = [pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"]), pytest.mark.parametrize("dtype", [BF16, FP16]),
       pytest.mark.parametrize("d", [64, 128]), pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])]


def every(test):
    for mark in ALL:
        test = mark(test)
    return test


def made(gpu, shape, dtype, d, tree, **kw):
    return Made(gpu, shape["lens"], shape["nodes"], shape["Hq"], shape["H"], d, 32, 16, dtype, tree=tree, **kw)


def empty_block(m, b, caches):
    """The last, partly filled block of sequence b as an append of zeros leaves it: scale 2^-118."""
    n = m.lens[b]
    page, first = m.table_list[b][(n - 1) // m.page], (n - 1) % m.page // 16 * 16
    for c, s in caches:
        c.view(torch.uint8)[page, :, first:(n - 1) % m.page + 1] = 0
        s[page, :, first // 16] = 2.0 ** -118


@every
def test_queries_of_zero(gpu, shape, dtype, d, tree):
    m = made(gpu, shape, dtype, d, tree)
    m.q[: m.T] = 0
    m.check()


@every
def test_one_tokens_queries_of_zero(gpu, shape, dtype, d, tree):
    m = made(gpu, shape, dtype, d, tree)
    at = serving_ref.offsets(m.nodes)
    for b, n in enumerate(m.nodes):
        for i in (0, n // 2, n - 1):
            was = m.q[at[b] + i].clone()
            m.q[at[b] + i] = 0
            m.check()
            m.q[at[b] + i] = was


@every
def test_queries_and_keys_of_zero(gpu, shape, dtype, d, tree):
    m = made(gpu, shape, dtype, d, tree)
    m.q[: m.T], m.k[: m.T] = 0, 0
    m.check()
    m.v[: m.T] = 0
    m.check()


@every
@pytest.mark.parametrize("size", [-20, -40, -100])
def test_tiny_queries_and_keys(gpu, shape, dtype, d, tree, size):
    m = made(gpu, shape, dtype, d, tree)
    m.q[: m.T] *= 2.0 ** size
    m.check()
    m.k[: m.T] *= 2.0 ** size
    m.check()


@every
def test_cached_blocks_of_zeros(gpu, shape, dtype, d, tree):
    for zero_q in (False, True):
        for of_k, of_v in ((True, False), (False, True), (True, True)):
            m = made(gpu, shape, dtype, d, tree)
            for b in (0, 2, 3):
                empty_block(m, b, [(m.kc, m.ks)] * of_k + [(m.vc, m.vs)] * of_v)
            if zero_q:
                m.q[: m.T] = 0
            m.check()


@every
def test_all_zero(gpu, shape, dtype, d, tree):
    """A warm-up: rows, cache and scales as such a call finds them. O is 0, the LSE the logarithm of how many are seen."""
    m = made(gpu, shape, dtype, d, tree)
    for x in (m.q, m.k, m.v, m.kc.view(torch.uint8), m.vc.view(torch.uint8)):
        x.zero_()
    for scale in (1.0, 2.0 ** -118):
        m.ks.fill_(scale)
        m.vs.fill_(scale)
        o, _ = m.check()
        assert bool((o[: m.T] == 0).all())
