"""The serving attention where a lane takes many steps an item: contexts and batches long enough that every
CTA gets a run of many key tiles, with keys that grow along a sequence, so that the running maximum
moves, for some of a warp's rows only.

Trees and decoding: K and V of a tile loaded in one go (few rows; d = 64, or pages of 16 tokens) and a slot
at a time. Prompts: items of two query tiles. Also one such shape in each of the library's test builds.
"""

import random

import pytest
import torch

import serving_ref as ref
from io_aware_exact_04_gb300 import _lib, api
from test_serving_gpu import Cache, ints, masks_of, normal, ok, rows_like

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def grow(rows, most):
    """Keys that grow along a sequence, up to `most` times their size."""
    n = rows.shape[0]
    return (rows.float() * torch.linspace(0.3, most, max(n, 1), device=rows.device)[:n, None, None]).to(rows.dtype)


def grown_cache(lens, hkv, page, d, dtype, device, most, seed=0, order="hpd"):
    c = Cache(lens, hkv, page, d, dtype, device, seed=seed, order=order)
    for b, n in enumerate(lens):
        k = grow(c.rows[b][0], most)
        c.rows[b] = torch.stack([k, c.rows[b][1]])
        for j in range(-(-n // page)):
            part = k[page * j:page * (j + 1)]
            c.kv[0, int(c.table[b, j]), :, :part.shape[0]] = part.transpose(0, 1)
    return c


def uneven(q, seed):
    """Queries of very different sizes: the maximum moves by more than the threshold for a few rows only."""
    r = random.Random(seed)
    f = torch.tensor([[r.choice([0.05, 0.2, 1.0, 2.0]) for _ in range(q.shape[1])] for _ in range(q.shape[0])], device=q.device)
    return (q.float() * f[:, :, None]).to(q.dtype)


def check(o, lse, want, T, q, v_rows):
    """Bounds as in serving_ref, and for fp16 the bits that P loses below 2^-23 of the largest: P is stored as
    2^9 p or more (relative to the row's reference maximum, which is at most the final one), off by at most half of
    the smallest step, 2^-25, so p by 2^-34; times the sum of |v| over the keys."""
    ro, rl, do, dl = want
    if q.dtype is torch.float16:
        do = do + 2.0 ** -34 * v_rows
    ref.assert_close(o, lse, (ro, rl, do, dl), T)


FEW = [(64, 16), (64, 32), (64, 64), (64, 128), (64, 256), (128, 16)]  # K and V of a tile in one go
FEW_APART = [(128, 32), (128, 64)]                                     # a slot at a time


def few_case(d, page, dtype, gpu, kind, seed, bad_pages=False):
    r = random.Random(seed)
    Hkv, G, B = 8, 2, 36
    lens = [r.choice([0, 1, 1100, 1152, 1153, r.randrange(900, 2600), r.randrange(900, 2600), r.randrange(900, 2600)])
            for _ in range(B)]
    nodes = [r.choice([1, 1, 1, 2, 3, 4, 5, 8]) for _ in range(B)]  # up to 8 and up to 16 rows
    nodes[3] = 0
    T = sum(nodes)
    q, k, v = rows_like("fused", T, G * Hkv, Hkv, d, dtype, gpu, seed=seed)
    q, k = uneven(q, seed), k * 4
    c = grown_cache(lens, Hkv, page, d, dtype, gpu, 5.0, seed=seed, order=r.choice(["hpd", "phd"]))
    table, ctx = c.table, c.ctx
    if bad_pages:  # pages of zeros, one in the middle of a tile's boxes and one at a sequence's end
        table = table.clone()
        rows = [x.clone() for x in c.rows]
        for b, n in enumerate(lens):
            if n == 0 or b % 3:
                continue
            for j, id_ in ((n // page // 2, 1 << 24), ((n - 1) // page, -5)):
                table[b, j] = id_
                rows[b][:, page * j:page * (j + 1)] = 0
        ctx = lambda b: (rows[b][0], rows[b][1])  # noqa: E731
    mask, seen = None, None
    if kind:
        words, bits, _ = masks_of(kind, nodes, seed)
        mask = torch.cat([ref.pack_bits(s, words) for s in bits]).to(gpu)
        seen = lambda b, n: bits[b][:, :n]  # noqa: E731
    cu = ints(ref.offsets(nodes), gpu)
    want = ref.forward(q, k, v, nodes, d ** -0.5, ctx=ctx, seen_nodes=seen)
    return dict(q=q, k=k, v=v, k_cache=c.kv[0], v_cache=c.kv[1], table=table, lens=c.lens, cu_nodes=cu, mask=mask), want, T


V_SUM = 2700 * 5.0  # above the sum of |v| over any row's keys: standard normals, 2608 of them at most


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", [None, "tree", "random"])
@pytest.mark.parametrize("d,page", FEW + FEW_APART)
def test_few_rows_over_many_tiles(gpu, d, page, kind, dtype):
    call, want, T = few_case(d, page, DTYPES[dtype], gpu, kind, seed=page + d)
    o, lse = api.forward_tree(**call)
    ok(gpu)
    check(o, lse, want, T, call["q"], V_SUM)
    for _ in range(3):
        o2, lse2 = api.forward_tree(**call, out=torch.full_like(o, float("nan")))
        assert torch.equal(o, o2) and torch.equal(lse, lse2), "another call differs"


@pytest.mark.parametrize("d,page", FEW + FEW_APART)
def test_few_rows_bad_pages(gpu, d, page):
    """Page ids outside the cache are pages of zeros, and recorded."""
    call, want, T = few_case(d, page, torch.bfloat16, gpu, None, seed=page + d, bad_pages=True)
    o, lse = api.forward_tree(**call)
    torch.cuda.synchronize(gpu)
    assert api.device_status(gpu)[0] == 6
    check(o, lse, want, T, call["q"], V_SUM)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", [None, "tree", "random"])
@pytest.mark.parametrize("d,page,Hq,Hkv", [(64, 16, 8, 8), (64, 64, 12, 4), (128, 32, 16, 4), (128, 128, 5, 5)])
def test_many_rows_over_many_tiles(gpu, d, page, Hq, Hkv, kind, dtype):
    """Drafts and further parts of prompts: items of one and of two query tiles."""
    r = random.Random(d + Hq)
    B = 10
    lens = [r.choice([0, 64, r.randrange(900, 2600), r.randrange(900, 2600)]) for _ in range(B)]
    nodes = [r.choice([1, 17, 40, 100, 130, 200, 333]) for _ in range(B)]
    T = sum(nodes)
    q, k, v = rows_like("fused", T, Hq, Hkv, d, DTYPES[dtype], gpu, seed=d)
    q, k = uneven(q, d), k * 4
    c = grown_cache(lens, Hkv, page, d, DTYPES[dtype], gpu, 5.0, seed=page)
    mask, seen = None, None
    if kind:
        words, bits, _ = masks_of(kind, nodes, 5)
        mask = torch.cat([ref.pack_bits(s, words) for s in bits]).to(gpu)
        seen = lambda b, n: bits[b][:, :n]  # noqa: E731
    o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, ints(ref.offsets(nodes), gpu), mask=mask)
    ok(gpu)
    check(o, lse, ref.forward(q, k, v, nodes, d ** -0.5, ctx=c.ctx, seen_nodes=seen), T, q, 3000 * 5.0)


# lengths that leave the second query tile of a pair whole, partial and missing
PAIR_LENS = [1000, 129, 1537, 64, 2048, 1, 999, 1090, 65, 1300, 0, 700, 1921, 191]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(16, 16), (16, 8), (15, 5)])
def test_prompts_in_pairs(gpu, Hq, Hkv, d, dtype):
    """Enough prompts that items take two query tiles (their key tiles together are several times the longest
    item's for every CTA)."""
    T = sum(PAIR_LENS)
    q, k, v = rows_like("fused", T, Hq, Hkv, d, DTYPES[dtype], gpu, seed=Hq + d)
    k = torch.cat([grow(x, 5.0) for x in k.split(PAIR_LENS)])
    q = uneven(q, 3)
    cu = ints(ref.offsets(PAIR_LENS), gpu)
    o, lse = api.forward_prompt(q, k, v, cu)
    ok(gpu)
    check(o, lse, ref.forward(q, k, v, PAIR_LENS, d ** -0.5), T, q, 2048 * 5.0)
    o2, lse2 = api.forward_prompt(q, k, v, cu, out=torch.full_like(o, float("nan")))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.fixture
def build(gpu, monkeypatch):
    def use(name):
        lib = _lib.load(name)
        monkeypatch.setattr(api, "_lib_fa", lambda: lib)
        api.device_status(gpu)
    return use


@pytest.mark.parametrize("d,page", [(64, 32), (128, 16)])
def test_debug_build(build, gpu, d, page):
    """No check of the bounds-checked build fires, and the results are right."""
    call, want, T = few_case(d, page, torch.float16, gpu, "tree", seed=3)
    build("libfa_debug.so")
    o, lse = api.forward_tree(**call)
    ok(gpu)
    check(o, lse, want, T, call["q"], V_SUM)


@pytest.mark.parametrize("d,page", [(64, 32), (128, 16)])
def test_copies_that_never_arrive(build, gpu, d, page):
    """Copies left out where K and V are loaded in one go: reported, and the context stays usable."""
    call, want, T = few_case(d, page, torch.bfloat16, gpu, None, seed=4)
    build("libfa_withhold.so")
    api.forward_tree(**call)
    torch.cuda.synchronize(gpu)
    code, detail = api.device_status(gpu)
    assert code == 5 and 60 <= detail[1] <= 72, detail
    build("libfa.so")
    o, lse = api.forward_tree(**call)
    ok(gpu)
    check(o, lse, want, T, call["q"], V_SUM)
