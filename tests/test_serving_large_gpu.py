"""The serving operators where an element's offset passes 31 and 32 bits, with many sequences, and inside
CUDA graphs.

Where the data lies does not enter the arithmetic: the same tokens in other pages, or in rows
further apart, give the same bits.
"""

import random

import pytest
import torch

import serving_ref as ref
from io_aware_exact_04_gb300 import api
from test_serving_gpu import Cache, ints, masks_of, normal, ok, rows_like

pytestmark = pytest.mark.gpu

FAR = 70000  # pages of 65536 elements: a plane of 4.6e9 elements


@pytest.fixture
def far_pool(gpu):
    """Two planes of 70000 pages of 8 heads, 64 tokens, d = 128; only the pages in use are written."""
    if torch.cuda.mem_get_info(gpu)[0] < 40 << 30:
        pytest.skip("needs 40 GB of free memory")
    yield torch.empty((2, FAR, 8, 64, 128), dtype=torch.bfloat16, device=gpu)
    torch.cuda.empty_cache()


def test_pages_far_apart(gpu, far_pool):
    """Append, attention, update and compaction with pages past 2^31 and 2^32 elements and bytes."""
    d, H, page, lens = 128, 8, 64, [130, 64, 200]
    near = normal(2, 16, H, page, d, dtype=torch.bfloat16, device=gpu)
    ids = [[0, 1, 2, -1], [3, -1, -1, -1], [4, 5, 6, 7]]
    far_of = [FAR - 1, 32768, 32769, 65535, 65536, 40000, 16384, 69000]
    far_ids = [[far_of[i] if i >= 0 else -1 for i in r] for r in ids]
    for i, f in enumerate(far_of):
        far_pool[:, f] = near[:, i]
    results = []
    for kv, table in ((near, ids), (far_pool, far_ids)):
        table, at = ints(sum(table, []), gpu).view(3, 4), ints(lens, gpu)
        q, k, v = rows_like("plain", 9, 16, H, d, torch.bfloat16, gpu, seed=3)
        cu = ints([0, 4, 4, 9], gpu)
        o, lse = api.forward_tree(q, k, v, kv[0], kv[1], table, at, cu)
        api.cache_append(k, v, kv[0], kv[1], table, at, cu)
        # slot 1 becomes the first 100 tokens of slot 2, and so gets a page of its own for the last 36
        grown = ints([134, 64, 205], gpu)
        info = api.cache_update(kv, table, grown, ints([0, 2, 2], gpu), ints([134, 100, 205], gpu))
        o1, lse1 = api.forward_tree(q[:3], k[:3], v[:3], kv[0], kv[1], table, grown, ints([0, 1, 2, 3], gpu))
        api.cache_compact(kv, table, grown)
        o2, lse2 = api.forward_tree(q[:3], k[:3], v[:3], kv[0], kv[1], table, grown, ints([0, 1, 2, 3], gpu))
        ok(gpu)
        assert info.tolist()[0] == 1 and grown.tolist() == [134, 100, 205]
        assert torch.equal(o1, o2) and torch.equal(lse1, lse2)
        used = {int(x) for row, n in zip(table.tolist(), (3, 2, 4)) for x in row[:n]}
        assert used == set(range(8))
        results.append((o, lse, o1, lse1))
    for x, y in zip(*results):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_far_apart(gpu, d):
    """Rows of q, k, v and o whose token stride takes them past 2^31 elements."""
    T, Hq, Hkv, stride = 150, 4, 2, 1 << 24
    if torch.cuda.mem_get_info(gpu)[0] < 40 << 30:
        pytest.skip("needs 40 GB of free memory")
    wide = torch.empty((T, stride), dtype=torch.float16, device=gpu)
    q, k, v = rows_like("plain", T, Hq, Hkv, d, torch.float16, gpu, seed=5)
    at, views = 0, []
    for x in (q, k, v, None):
        H = Hq if x is None else x.shape[1]
        views.append(wide[:, at:at + H * d].unflatten(1, (H, d)))
        at += H * d
        if x is not None:
            views[-1].copy_(x)
    cu = ints([0, 20, T], gpu)
    want, lse = api.forward_prompt(q, k, v, cu)
    got, glse = api.forward_prompt(*views[:3], cu, out=views[3])
    ok(gpu)
    assert torch.equal(got, want) and torch.equal(glse, lse)
    c = Cache([50, 3], Hkv, 16, d, torch.float16, gpu, width=20)
    want, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu)
    got, glse = api.forward_tree(*views[:3], c.kv[0], c.kv[1], c.table, c.lens, cu, out=views[3])
    ok(gpu)
    assert torch.equal(got, want) and torch.equal(glse, lse)
    table = torch.arange(40, dtype=torch.int32, device=gpu).view(2, 20)
    pools = [torch.zeros((2, 40, Hkv, 16, d), dtype=torch.float16, device=gpu) for _ in range(2)]
    for pool, (kk, vv) in zip(pools, ((k, v), views[1:3])):
        api.cache_append(kk, vv, pool[0], pool[1], table, ints([0, 0], gpu), cu)
    ok(gpu)
    assert torch.equal(pools[0], pools[1]) and bool(pools[0].any())
    del wide, views, got
    torch.cuda.empty_cache()


def test_prompt_replayed_with_other_lengths(gpu):
    """A captured call takes its lengths from the device at every replay."""
    d, T = 128, 700
    q, k, v = rows_like("fused", T, 8, 2, d, torch.bfloat16, gpu, seed=6)
    cu = ints([0, 1, 2, 3], gpu)
    api.forward_prompt(q, k, v, cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = api.forward_prompt(q, k, v, cu)
    for lens in ([700, 0, 0], [129, 0, 571], [1, 300, 200]):
        cu.copy_(ints(ref.offsets(lens), gpu))
        graph.replay()
        ok(gpu)
        ref.assert_close(o, lse, ref.forward(q, k, v, lens, d ** -0.5), sum(lens))


def test_pool_replayed_with_other_slots(gpu):
    """A serving step's append, update and compaction in one graph, replayed with other slots and
    lengths, against the same calls one by one."""
    d, H, page = 64, 2, 16
    start = Cache([40, 0, 17, 100], H, page, d, torch.float16, gpu, width=12, extra=30)
    k, v = normal(6, H, d, dtype=torch.float16, device=gpu), normal(6, H, d, dtype=torch.float16, device=gpu)

    def step(kv, table, lens, src, new, at, cu):
        first = api.cache_update(kv, table, lens, src, new)
        api.cache_append(k, v, kv[0], kv[1], table, at, cu)
        return first, api.cache_compact(kv, table, lens)

    def state():
        return [start.kv.clone(), start.table.clone(), start.lens.clone()] + [ints(x, gpu) for x in (
            [0, 1, 2, 3], [40, 0, 17, 100], [39, 0, 16, 99], [0, 1, 1, 2, 3])]

    captured = state()
    step(*captured)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        infos = step(*captured)
    for src, new, cu in (([3, 3, 0, 2], [90, 70, 42, 20], [0, 2, 3, 5, 6]), ([1, 2, 2, 0], [0, 17, 30, 40], [0, 0, 1, 4, 6]),
                         ([0, 1, 2, 3], [0, 0, 0, 192], [0, 0, 0, 0, 6])):
        plain = state()
        taken = [max(0, n - (y - x)) for n, x, y in zip(new, cu, cu[1:])]
        for t, x in zip(plain[3:], (src, new, taken, cu)):
            t.copy_(ints(x, gpu))
        for t, x in zip(captured, plain):
            t.copy_(x)
        want = step(*plain)
        graph.replay()
        ok(gpu)
        for x, y in zip(captured, plain):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))  # (unused pages hold NaN)
        for x, y in zip(infos, want):
            assert torch.equal(x, y)
        assert plain[2].tolist() == new


@pytest.mark.parametrize("count,Hq,Hkv,d", [(129, 2, 1, 64), (300, 6, 3, 128), (1000, 1, 1, 64), (200, 20, 5, 128)])
def test_many_sequences(gpu, count, Hq, Hkv, d):
    """Hundreds of sequences: mostly short, some empty, a few long."""
    r = random.Random(count)
    lens = [r.choice([0, 1, r.randrange(2, 40), r.randrange(2, 40), 129]) for _ in range(count)]
    for b in (0, count // 2, count - 1):
        lens[b] = r.randrange(700, 900)
    T = sum(lens)
    q, k, v = rows_like("fused", T, Hq, Hkv, d, torch.bfloat16, gpu, seed=count)
    cu = ints(ref.offsets(lens), gpu)
    o, lse = api.forward_prompt(q, k, v, cu)
    ok(gpu)
    ref.assert_close(o, lse, ref.forward(q, k, v, lens, d ** -0.5), T)
    c = Cache([r.choice([0, r.randrange(300)]) for _ in lens], Hkv, 32, d, torch.bfloat16, gpu)
    o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu)
    ok(gpu)
    ref.assert_close(o, lse, ref.forward(q, k, v, lens, d ** -0.5, ctx=c.ctx), T)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes,Hq,Hkv", [(1, 7, 1), (1, 16, 2), (1, 9, 1), (8, 2, 2), (9, 1, 1), (5, 3, 1), (16, 1, 1), (17, 1, 1),
                                          (4, 16, 4), (1, 17, 1), (2, 16, 2)])
def test_few_rows(gpu, nodes, Hq, Hkv, d, dtype):
    """Around 8 and 16 rows a key/value head; scores that grow along the keys, so that the running
    maximum moves; trees and chains."""
    lens = [0, 1, 63, 64, 65, 127, 129, 400, 1000]
    T = nodes * len(lens)
    q, k, v = rows_like("fused", T, Hq, Hkv, d, dtype, gpu, seed=nodes)
    c = Cache(lens, Hkv, 32, d, dtype, gpu, seed=d)
    for b, n in enumerate(lens):  # keys grow tenfold along a sequence
        grown = (c.rows[b][0].float() * torch.linspace(0.5, 5, max(n, 1), device=gpu)[:n, None, None]).to(dtype)
        c.rows[b] = torch.stack([grown, c.rows[b][1]])
        for j in range(-(-n // 32)):
            part = grown[32 * j:32 * j + 32]
            c.kv[0, int(c.table[b, j]), :, :part.shape[0]] = part.transpose(0, 1)
    cu = ints(ref.offsets([nodes] * len(lens)), gpu)
    o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu)
    ok(gpu)
    ref.assert_close(o, lse, ref.forward(q, k, v, [nodes] * len(lens), d ** -0.5, ctx=c.ctx), T)
    for kind in ("tree", "random"):
        words, bits, _ = masks_of(kind, [nodes] * len(lens), 3)
        mask = torch.cat([ref.pack_bits(s, words) for s in bits]).to(gpu)
        o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu, mask=mask)
        ok(gpu)
        ref.assert_close(o, lse, ref.forward(q, k, v, [nodes] * len(lens), d ** -0.5, ctx=c.ctx,
                                             seen_nodes=lambda b, n: bits[b][:, :n]), T)
