"""Attention over a cache in 8 bits, against the definition in 64 bits."""

import math

import pytest
import torch

from io_aware_exact_04_gb300 import api
from tests import cache8_ref as ref
from tests import serving_ref

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
BF16, FP16 = torch.bfloat16, torch.float16


def ints(x, gpu):
    return torch.tensor(x, dtype=torch.int32, device=gpu)


class Made:
    """Inputs of one call; everything behind a sequence's length, in the pages and among the rows, is poisoned."""

    def __init__(self, gpu, lens, nodes, Hq, H, d, page, block, dtype, seed=0, tree=False, tail=5, spread=2.0, words=None):
        g = torch.Generator(device=gpu).manual_seed(seed * 1000 + d + Hq)
        self.gpu, self.lens, self.nodes, self.page, self.dtype = gpu, lens, nodes, page, dtype
        self.scale = 1.0 / math.sqrt(d)
        T = sum(nodes) + tail
        self.T = sum(nodes)
        self.q, self.k, self.v = (torch.randn((T, h, d), generator=g, device=gpu).to(dtype) for h in (Hq, H, H))
        for x in (self.q, self.k, self.v):
            x[self.T:] = math.nan
        need = [-(-n // page) for n in lens]
        pool = sum(need) + 2
        ids = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table_list = [[ids.pop() for _ in range(n)] + [-1] * (max(need) + 1 - n) for n in need]
        self.table = ints(self.table_list, gpu)
        self.kc, self.vc, self.ks, self.vs = [], [], [], []
        size = torch.exp2(spread * torch.randn((pool, H, page // block, 1, 1), generator=g, device=gpu))
        out = []
        for which in range(2):
            x = torch.randn((pool, H, page // block, block, d), generator=g, device=gpu) * (size if which else 1.0)
            out.append(ref.quantised(x.flatten(2, 3), page // block))
        (self.kc, self.ks), (self.vc, self.vs) = out
        # 0x7f is NaN: what lies behind a length must not reach a result; nor do the scales of blocks without a token
        used = torch.zeros((pool, page), dtype=torch.bool, device=gpu)
        for b, n in enumerate(lens):
            for j, p in enumerate(self.table_list[b][: need[b]]):
                used[p, : min(page, n - j * page)] = True
        for c in (self.kc, self.vc):
            c.view(torch.uint8).masked_fill_(~used[:, None, :, None], 0x7F)
        any_used = used.unflatten(1, (page // block, block)).any(-1)
        for s in (self.ks, self.vs):
            s.masked_fill_(~any_used[:, None], math.nan)
        self.cu = ints(serving_ref.offsets(nodes), gpu)
        self.len_t = ints(lens, gpu)
        self.mask = self.seen = None
        if tree:
            r = torch.Generator().manual_seed(seed + 7)
            self.words = words or max(1, -(-max(nodes) // 32))
            bits = torch.zeros((T, self.words * 32), dtype=torch.bool)
            self.per = []
            at = 0
            for n in nodes:
                x = torch.rand((n, n), generator=r) < 0.5  # any bits, not a tree's alone; some rows see nothing
                x[: n // 3] = False
                self.per.append(x.to(gpu))
                bits[at:at + n, :n] = x
                bits[at:at + n, n:] = True  # behind the sequence's nodes: count as not set
                at += n
            w = (bits.reshape(T, self.words, 32).long() << torch.arange(32)).sum(-1)
            self.mask = torch.where(w >= 1 << 31, w - (1 << 32), w).int().to(gpu)
            self.seen = lambda b, n: self.per[b]

    def call(self, **kw):
        return api.forward_tree(self.q, self.k, self.v, self.kc, self.vc, self.table, self.len_t, self.cu, mask=self.mask,
                                scale=self.scale, k_scale=self.ks, v_scale=self.vs, **kw)

    def want(self):
        k, v = (ref.dequantised(c, s).nan_to_num(0.0) for c, s in ((self.kc, self.ks), (self.vc, self.vs)))
        rows = lambda b: (serving_ref.rows_of_cache(k, self.table, b, self.lens[b]),
                          serving_ref.rows_of_cache(v, self.table, b, self.lens[b]))
        return serving_ref.forward(self.q[: self.T], self.k[: self.T], self.v[: self.T], self.nodes, self.scale, ctx=rows,
                                   seen_nodes=self.seen)

    def check(self, got=None):
        o, lse = self.call() if got is None else got
        wo, wl, do, dl = self.want()
        assert api.device_status(self.gpu)[0] == 0
        serving_ref.assert_close(o[: self.T], lse[:, : self.T], (wo, wl, do, dl), self.T)
        return o, lse


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("lens,nodes,Hq,H,d,page,block", [
    ([1], [1], 1, 1, 64, 16, 16),
    ([0, 1, 127, 128, 129], [1, 1, 1, 1, 1], 2, 1, 128, 16, 16),
    ([700, 33, 0, 256, 300], [1, 0, 2, 1, 3], 12, 12, 64, 32, 16),
    ([1000, 90, 513], [1, 4, 2], 8, 2, 128, 64, 64),
    ([2000, 17], [1, 1], 16, 1, 128, 128, 32),
    ([600, 40], [5, 7], 15, 3, 64, 256, 128),
    ([300, 31], [9, 20], 14, 2, 128, 64, 32),
    ([257], [64], 4, 1, 64, 256, 256),
    ([130, 5], [40, 33], 40, 5, 128, 32, 32),
    ([64], [3], 128, 1, 64, 64, 16),
])
def test_chains(gpu, dtype, lens, nodes, Hq, H, d, page, block):
    Made(gpu, lens, nodes, Hq, H, d, page, block, dtype, seed=len(lens)).check()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("lens,nodes,Hq,H,d,page,block", [
    ([0], [3], 1, 1, 64, 16, 16),
    ([0, 0, 200], [6, 1, 9], 4, 2, 128, 32, 32),
    ([333, 128], [7, 16], 12, 12, 64, 16, 16),
    ([900, 10, 64], [33, 64, 5], 8, 2, 128, 64, 64),
    ([100], [100], 5, 1, 128, 128, 64),
])
def test_trees_and_rows_that_see_nothing(gpu, dtype, lens, nodes, Hq, H, d, page, block):
    m = Made(gpu, lens, nodes, Hq, H, d, page, block, dtype, seed=3, tree=True)
    o, lse = m.check()
    if lens[0] == 0:  # the first nodes see nothing at all
        n = nodes[0] // 3
        assert bool((o[:n] == 0).all()) and bool((lse[:, :n] == -math.inf).all())


def test_random_shapes(gpu):
    import random
    r = random.Random(11)
    for seed in range(24):
        H = r.choice([1, 2, 3])
        G = r.choice([1, 2, 3, 5, 8, 16, 33])
        page = r.choice([16, 32, 64, 128, 256])
        block = r.choice([b for b in (16, 32, 64, 128, 256) if b <= page])
        seqs = r.randrange(1, 9)
        lens = [r.choice([0, r.randrange(1, 40), r.randrange(1, 1500)]) for _ in range(seqs)]
        nodes = [r.choice([0, 1, 1, r.randrange(1, 12), r.randrange(1, 70)]) for _ in range(seqs)]
        if not any(nodes):
            nodes[0] = 1
        Made(gpu, lens, nodes, G * H, H, r.choice([64, 128]), page, block, r.choice([BF16, FP16]), seed=seed,
             tree=r.random() < 0.5).check()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("most", [3, 14, 40])
def test_many_items_of_both_kinds(gpu, dtype, d, most):
    """More items than CTAs, some of one lane's rows and some of two, in turn: every ring goes round several times,
    with slots that one lane skips."""
    import random
    r = random.Random(most)
    lens = [r.choice([0, 5, 130, 300, r.randrange(1, 700)]) for _ in range(40)]
    nodes = [r.choice([1, 2, most, r.randrange(0, most + 1)]) for _ in range(40)]
    m = Made(gpu, lens, nodes, 24, 6, d, 64, 32, dtype, seed=most, tree=most == 14)
    first = m.check()
    for _ in range(3):  # no atomics, one order of sums: the same bits
        again = m.call()
        assert all(torch.equal(x[..., : m.T] if x.dim() == 2 else x[: m.T], y[..., : m.T] if y.dim() == 2 else y[: m.T])
                   for x, y in zip(first, again))


def test_refusals(gpu):
    m = Made(gpu, [40, 3], [1, 1], 4, 2, 64, 32, 16, BF16)
    need = api._tree_workspace(gpu.index, 64, "fa_forward_tree_8bit")
    m.call(workspace=torch.empty(need, dtype=torch.uint8, device=gpu))
    with pytest.raises(RuntimeError):
        m.call(workspace=torch.empty(need - 1, dtype=torch.uint8, device=gpu))
    for name, bad in (("ks", None), ("vs", m.vs[:, :, :1]), ("ks", m.ks.double()), ("kc", m.kc.view(torch.uint8)),
                      ("vc", m.vc[:, :1]), ("kc", m.kc.to(BF16)), ("q", m.q.float()), ("table", m.table[:1])):
        was = getattr(m, name)
        setattr(m, name, bad)
        with pytest.raises(ValueError):
            m.call()
        setattr(m, name, was)
    m.check()


@pytest.mark.parametrize("Hq,H,d,dtype", [(12, 12, 64, FP16), (32, 8, 128, BF16), (16, 2, 128, FP16), (20, 4, 64, BF16)])
def test_many_calls_in_a_row(gpu, Hq, H, d, dtype):
    """Long contexts, many items, calls that follow each other without a wait, from a cold start: every product may lag
    behind by as much as the buffers allow. No wait runs out, and all calls give the same bits."""
    lens = [5000 - 37 * i for i in range(64)]
    m = Made(gpu, lens, [1] * 64, Hq, H, d, 32, 16, dtype, seed=2)
    outs = [m.call() for _ in range(30)]
    assert api.device_status(gpu)[0] == 0
    for o, lse in outs[1:]:
        assert torch.equal(o[: m.T], outs[0][0][: m.T]) and torch.equal(lse[:, : m.T], outs[0][1][:, : m.T])
    m.check(outs[-1])
