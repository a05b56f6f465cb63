"""Prompts, drafted trees over a cache in pages, and the cache's own work, against plain 64-bit forms."""

import math
import random

import pytest
import torch

import serving_ref as ref
from io_aware_exact_04_gb300 import api

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]


def normal(*shape, dtype, device, seed=0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=device, dtype=torch.float32).to(dtype)


def ints(x, device):
    return torch.tensor(x, dtype=torch.int32, device=device)


def ok(device):
    torch.cuda.synchronize(device)
    code, detail = api.device_status(device)
    assert code == 0, f"device status {detail}"


def rows_like(layout, T, Hq, Hkv, d, dtype, device, seed=0):
    """q, k, v in a layout: contiguous, views of one projection, or views of head-major tensors."""
    if layout == "fused":
        x = normal(T, Hq + 2 * Hkv, d, dtype=dtype, device=device, seed=seed)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if layout == "heads":
        x = normal(Hq + 2 * Hkv, T, d, dtype=dtype, device=device, seed=seed).transpose(0, 1)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    return tuple(normal(T, H, d, dtype=dtype, device=device, seed=seed + i) for i, H in enumerate((Hq, Hkv, Hkv)))


class Cache:
    """A pool in pages with random page ids; what no token uses holds NaN."""

    def __init__(self, lens, hkv, page, d, dtype, device, extra=3, width=None, seed=0, order="hpd"):
        r = random.Random(seed)
        pages = [-(-n // page) for n in lens]
        self.width = max(1, max(pages, default=0)) + 1 if width is None else width
        pool = sum(pages) + extra
        ids = r.sample(range(pool), pool)
        self.table = torch.full((len(lens), self.width), -7, dtype=torch.int32)
        shape = (2, pool, hkv, page, d) if order == "hpd" else (2, pool, page, hkv, d)
        kv = torch.full(shape, float("nan"), dtype=dtype, device=device)
        self.kv = kv if order == "hpd" else kv.transpose(2, 3)
        self.rows = []
        for b, n in enumerate(lens):
            mine = [ids.pop() for _ in range(pages[b])]
            self.table[b, : len(mine)] = torch.tensor(mine, dtype=torch.int32)
            x = normal(2, n, hkv, d, dtype=dtype, device=device, seed=seed * 1000 + b)
            self.rows.append(x)
            for j, p in enumerate(mine):
                part = x[:, j * page:(j + 1) * page]
                self.kv[:, p, :, : part.shape[1]] = part.transpose(1, 2)
        self.table = self.table.to(device)
        self.lens = ints(lens, device)

    def ctx(self, b):
        return self.rows[b][0], self.rows[b][1]


# ------------------------------------------------------------------------------------------------ prompts
PROMPTS = [
    # lens, Hq, Hkv, d, layout
    ([1], 1, 1, 64, "plain"),
    ([3, 0, 1], 2, 1, 64, "plain"),
    ([0, 127, 128, 129, 0], 4, 4, 64, "fused"),
    ([130, 1, 257], 6, 2, 128, "fused"),
    ([300], 5, 1, 128, "heads"),
    ([64, 65, 511, 2], 8, 1, 64, "heads"),
    ([700, 33], 7, 1, 128, "plain"),
    ([1500], 16, 1, 64, "plain"),
    ([40, 9], 128, 1, 128, "plain"),
    ([2, 1], 100, 1, 64, "plain"),
    ([1100, 1, 0, 260], 12, 12, 64, "fused"),
    ([2049], 4, 2, 128, "plain"),
    ([17] * 70, 3, 3, 64, "plain"),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("lens,Hq,Hkv,d,layout", PROMPTS)
def test_prompt(gpu, lens, Hq, Hkv, d, layout, dtype):
    T = sum(lens)
    q, k, v = rows_like(layout, T, Hq, Hkv, d, dtype, gpu, seed=5)
    cu = ints(ref.offsets(lens), gpu)
    o, lse = api.forward_prompt(q, k, v, cu)
    ok(gpu)
    want = ref.forward(q, k, v, lens, 1 / math.sqrt(d))
    ref.assert_close(o, lse, want, T)
    o2, lse2 = api.forward_prompt(q, k, v, cu, lse=False)
    assert lse2 is None and torch.equal(o, o2), "a second call differs"


def test_prompt_agrees_with_equal_heads(gpu):
    """The packed forward for equal heads and this one compute the same thing."""
    lens, H, d = [200, 77, 384], 4, 128
    T = sum(lens)
    q, k, v = (normal(H, T, d, dtype=torch.bfloat16, device=gpu, seed=i) for i in range(3))
    cu = ints(ref.offsets(lens), gpu)
    o1, l1 = api.forward_varlen(q, k, v, cu, max(lens), causal=True)
    o2, l2 = api.forward_prompt(q.transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1), cu)
    ok(gpu)
    assert float((l1 - l2).abs().max()) < 1e-5
    assert float((o1.transpose(0, 1).float() - o2.float()).abs().max()) <= 2 ** -6


def test_prompt_padding_and_foreign_rows(gpu):
    """Rows behind the last sequence stay as they were; NaN there and in other sequences' rows stays there."""
    lens, Hq, Hkv, d, pad = [70, 200, 30], 4, 2, 128, 41
    T = sum(lens) + pad
    q, k, v = (x.clone() for x in rows_like("plain", T, Hq, Hkv, d, torch.bfloat16, gpu))
    for x in (q, k, v):
        x[270:] = float("nan")  # the third sequence and the padding
    out = torch.full((T, Hq, d), 3.0, dtype=torch.bfloat16, device=gpu)
    lse = torch.full((Hq, T), 5.0, device=gpu)
    api.forward_prompt(q, k, v, ints(ref.offsets(lens), gpu), out=out, lse=lse)
    ok(gpu)
    want = ref.forward(q[:270], k[:270], v[:270], lens[:2], 1 / math.sqrt(d))
    ref.assert_close(out, lse, want, 270)
    assert torch.isnan(out[270:300].float()).all()
    assert (out[300:] == 3.0).all() and (lse[:, 300:] == 5.0).all()


def test_prompt_large_scores(gpu):
    """Scores of several hundred: the running maximum moves, nothing overflows."""
    lens, d = [400, 130], 64
    T = sum(lens)
    q, k, v = rows_like("plain", T, 4, 2, d, torch.bfloat16, gpu, seed=3)
    k = k * torch.linspace(0.1, 12, T, device=gpu, dtype=torch.bfloat16)[:, None, None]
    o, lse = api.forward_prompt(q * 4, k, v, ints(ref.offsets(lens), gpu), scale=0.7)
    ok(gpu)
    ref.assert_close(o, lse, ref.forward(q * 4, k, v, lens, 0.7), T)


# ------------------------------------------------------------------------------------------------ trees
TREES = [
    # ctx lens, nodes, Hq, Hkv, d, page, mask
    ([1], [1], 1, 1, 64, 16, None),
    ([0, 5, 128], [1, 1, 1], 4, 1, 64, 16, None),
    ([127, 129, 0, 300], [1, 0, 2, 1], 8, 2, 128, 32, None),
    ([700, 1], [7, 5], 12, 12, 64, 16, "tree"),
    ([0, 0], [9, 1], 6, 3, 128, 64, "tree"),
    ([1000, 513, 77], [26, 40, 0], 8, 2, 128, 64, "tree"),
    ([515, 130], [64, 33], 16, 4, 128, 128, "tree"),
    ([300, 2000], [130, 70], 4, 4, 64, 256, "tree"),
    ([0, 10], [6, 300], 3, 1, 128, 16, "random"),
    ([257], [37], 5, 1, 64, 32, "random"),
    ([4000], [1], 32, 4, 128, 64, None),
    ([3900], [3], 7, 1, 128, 256, None),
    ([90, 16, 0], [300, 513, 129], 4, 2, 64, 16, None),
    ([20], [5], 128, 1, 128, 16, "tree"),
    ([9] * 40, [2] * 40, 2, 2, 64, 16, "random"),
    ([1500, 8, 700] * 5, [1] * 15, 4, 2, 128, 64, None),
]


def masks_of(kind, nodes, seed=1):
    r = random.Random(seed)
    words = max(1, -(-max(nodes) // 32))
    seen, parents = [], []
    for n in nodes:
        p = [-1 if i == 0 or r.random() < 0.05 else r.randrange(max(0, i // 2 - 3), i) for i in range(n)]
        parents += p
        if kind == "random":  # any bits, some rows empty, bits past the nodes set too
            s = torch.tensor([[r.random() < 0.5 for _ in range(32 * words)] for _ in range(n)]).reshape(n, 32 * words)
            s[::3] = False
            seen.append(s)
        else:
            seen.append(ref.ancestors(p))
    return words, seen, parents


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("lens,nodes,Hq,Hkv,d,page,kind", TREES)
def test_tree(gpu, lens, nodes, Hq, Hkv, d, page, kind, dtype):
    T = sum(nodes)
    q, k, v = rows_like("fused" if d == 128 else "plain", T, Hq, Hkv, d, dtype, gpu, seed=2)
    c = Cache(lens, Hkv, page, d, dtype, gpu, seed=4, order="hpd" if page < 64 else "phd")
    cu = ints(ref.offsets(nodes), gpu)
    mask, seen = None, None
    if kind is not None:
        words, bits, parents = masks_of(kind, nodes)
        mask = torch.cat([ref.pack_bits(s, words) for s in bits]).to(gpu)
        if kind == "tree":
            made = api.tree_mask(ints(parents, gpu), cu, words)
            assert torch.equal(made, mask)
        seen = lambda b, n: bits[b][:, :n]  # noqa: E731
    o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu, mask=mask)
    ok(gpu)
    ref.assert_close(o, lse, ref.forward(q, k, v, nodes, 1 / math.sqrt(d), ctx=c.ctx, seen_nodes=seen), T)
    o2, lse2 = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu, mask=mask)
    assert torch.equal(o, o2) and torch.equal(lse, lse2), "a second call differs"


def test_tree_over_few_mask_words(gpu):
    """Nodes past the mask's words are not seen; every node still has its row."""
    nodes, d = [50], 64
    q, k, v = rows_like("plain", 50, 2, 1, d, torch.bfloat16, gpu)
    c = Cache([100], 1, 16, d, torch.bfloat16, gpu)
    full = torch.ones((50, 32), dtype=torch.bool)
    o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, ints([0, 50], gpu),
                              mask=ref.pack_bits(full, 1).to(gpu))
    ok(gpu)
    seen = torch.zeros((50, 50), dtype=torch.bool)
    seen[:, :32] = True
    ref.assert_close(o, lse, ref.forward(q, k, v, nodes, 1 / 8, ctx=c.ctx, seen_nodes=lambda b, n: seen), 50)


def test_tree_empty_rows(gpu):
    """No context and no bits: O = 0, LSE = -inf, beside a sequence that sees everything."""
    nodes, d = [3, 4], 128
    q, k, v = rows_like("plain", 7, 4, 2, d, torch.float16, gpu)
    c = Cache([0, 40], 2, 16, d, torch.float16, gpu)
    seen = [torch.zeros((3, 3), dtype=torch.bool), torch.ones((4, 4), dtype=torch.bool)]
    mask = torch.cat([ref.pack_bits(s, 1) for s in seen]).to(gpu)
    o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, ints([0, 3, 7], gpu), mask=mask)
    ok(gpu)
    assert (o[:3] == 0).all() and torch.isneginf(lse[:, :3]).all()
    ref.assert_close(o, lse, ref.forward(q, k, v, nodes, d ** -0.5, ctx=c.ctx, seen_nodes=lambda b, n: seen[b]), 7)


def test_tree_padding(gpu):
    """More slots than sequences have tokens for, rows behind the last one, slots whose table row is garbage."""
    nodes, d, T = [2, 0, 3], 64, 9
    q, k, v = (x.clone() for x in rows_like("plain", T, 4, 2, d, torch.bfloat16, gpu))
    c = Cache([50, 60, 200], 2, 32, d, torch.bfloat16, gpu)
    c.table[1] = 1 << 30
    lens = ints([50, -9, 200], gpu)  # slot 1 has no nodes: neither its length nor its pages are looked at
    for x in (q, k, v):
        x[5:] = float("nan")
    out = torch.full((T, 4, d), 3.0, dtype=torch.bfloat16, device=gpu)
    lse = torch.full((4, T), 5.0, device=gpu)
    api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, lens, ints([0, 2, 2, 5], gpu), out=out, lse=lse)
    ok(gpu)
    ref.assert_close(out, lse, ref.forward(q[:5], k[:5], v[:5], nodes, 1 / 8, ctx=c.ctx), 5)
    assert (out[5:] == 3.0).all() and (lse[:, 5:] == 5.0).all()


def test_tree_replayed_with_other_lengths(gpu):
    """Two captured calls, each replayed with other lengths, pages and nodes than it was captured with."""
    d, page, H = 128, 32, 4
    c = Cache([600, 40, 900], 2, page, d, torch.bfloat16, gpu, width=40)
    T = 12
    q, k, v = rows_like("plain", T, H, 2, d, torch.bfloat16, gpu, seed=9)
    calls = []
    for _ in range(2):
        lens, cu = ints([1, 1, 1], gpu), ints([0, 1, 2, 3], gpu)
        table = torch.zeros_like(c.table)
        api.forward_tree(q, k, v, c.kv[0], c.kv[1], table, lens, cu)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], table, lens, cu)
        calls.append((graph, table, lens, cu, o, lse))
    for (graph, table, lens, cu, o, lse), nodes in zip(calls, ([5, 0, 7], [1, 10, 1])):
        table.copy_(c.table)
        lens.copy_(c.lens)
        cu.copy_(ints(ref.offsets(nodes), gpu))
    for graph, *_ in calls:
        graph.replay()
    ok(gpu)
    for (graph, table, lens, cu, o, lse), nodes in zip(calls, ([5, 0, 7], [1, 10, 1])):
        ref.assert_close(o, lse, ref.forward(q, k, v, nodes, d ** -0.5, ctx=c.ctx), sum(nodes))


def test_tree_on_two_streams(gpu):
    """Calls on two streams at once, each with its own workspace."""
    d = 64
    c = Cache([3000, 100], 2, 16, d, torch.float16, gpu)
    q, k, v = rows_like("plain", 8, 8, 2, d, torch.float16, gpu)
    cu = ints([0, 4, 8], gpu)
    want, lw = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu)
    streams = [torch.cuda.Stream(gpu) for _ in range(2)]
    torch.cuda.synchronize(gpu)
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu))
    ok(gpu)
    for o, lse in got:
        assert torch.equal(o, want) and torch.equal(lse, lw)


def test_tree_bad_device_values(gpu):
    """Lengths past the table, page ids outside the cache, offsets that decrease: recorded, nothing else read."""
    d = 64
    q, k, v = rows_like("plain", 2, 2, 1, d, torch.bfloat16, gpu)
    c = Cache([40, 40], 1, 16, d, torch.bfloat16, gpu, width=3)
    cu = ints([0, 1, 2], gpu)
    table = c.table.clone()
    table[0, 1] = 1 << 20
    table[1, 0] = -3
    o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], table, c.lens, cu)
    torch.cuda.synchronize(gpu)
    assert api.device_status(gpu)[0] == 6

    def ctx(b):  # those pages are pages of zeros
        x = c.rows[b].clone()
        x[:, 16:32] = 0 if b == 0 else x[:, 16:32]
        x[:, :16] = 0 if b == 1 else x[:, :16]
        return x[0], x[1]

    ref.assert_close(o, lse, ref.forward(q, k, v, [1, 1], 1 / 8, ctx=ctx), 2)
    c2 = Cache([48, 40], 1, 16, d, torch.bfloat16, gpu, width=3)
    o, lse = api.forward_tree(q, k, v, c2.kv[0], c2.kv[1], c2.table, ints([5000, -4], gpu), cu)
    torch.cuda.synchronize(gpu)
    assert api.device_status(gpu)[0] == 6
    ref.assert_close(o, lse, ref.forward(q, k, v, [1, 1], 1 / 8, ctx=lambda b: [x[: 48 * (1 - b)] for x in c2.ctx(b)]), 2)
    for bad in ([0, 2, 1], [0, 1, 900], [-5, 1, 2]):
        api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, ints(bad, gpu))
        torch.cuda.synchronize(gpu)
        assert api.device_status(gpu)[0] == 6, bad
        api.forward_prompt(q, k, v, ints(bad, gpu))
        torch.cuda.synchronize(gpu)
        assert api.device_status(gpu)[0] == 6, bad


def test_tree_mask_bad_parents(gpu):
    cu = ints([0, 4, 6], gpu)
    m = api.tree_mask(ints([-1, 0, 2, 1, -5, 7], gpu), cu, 1)
    torch.cuda.synchronize(gpu)
    assert api.device_status(gpu)[0] == 6
    assert m[:, 0].tolist() == [1, 3, 4, 1 | 2 | 8, 1, 2]
    m = api.tree_mask(ints([-1] + list(range(39)), gpu), ints([0, 40], gpu), 1)
    torch.cuda.synchronize(gpu)
    assert api.device_status(gpu)[0] == 6
    assert m[35, 0].item() == -1 and m[3, 0].item() == 15


# ------------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("lens,new,Hkv,d,page,pick,order", [
    ([0], [1], 1, 64, 16, False, "hpd"),
    ([5, 0, 31, 64], [1, 0, 40, 3], 2, 128, 32, False, "hpd"),
    ([127, 3], [130, 7], 3, 64, 64, True, "phd"),
    ([10] * 50, [3] * 50, 8, 128, 16, True, "hpd"),
    ([100], [700], 5, 128, 256, False, "phd"),
])
def test_append(gpu, lens, new, Hkv, d, page, pick, order, dtype):
    c = Cache([a + b for a, b in zip(lens, new)], Hkv, page, d, dtype, gpu, order=order)
    T = sum(new)
    n = 2 * T + 5 if pick else T + 4  # rows behind the last sequence belong to nobody
    k, v = rows_like("fused", n, 1, Hkv, d, dtype, gpu, seed=8)[1:]
    rows = ints(random.Random(3).sample(range(n), T), gpu) if pick else None
    want = c.kv.clone()
    at = ref.offsets(new)
    for b in range(len(lens)):
        for i in range(new[b]):
            pos, row = lens[b] + i, int(rows[at[b] + i]) if pick else at[b] + i
            want[0, c.table[b, pos // page], :, pos % page] = k[row]
            want[1, c.table[b, pos // page], :, pos % page] = v[row]
    api.cache_append(k, v, c.kv[0], c.kv[1], c.table, ints(lens, gpu), ints(at, gpu), rows=rows)
    ok(gpu)
    assert torch.equal(c.kv.nan_to_num(77.0), want.nan_to_num(77.0))


def test_append_bad_offsets(gpu):
    """Recorded; the tokens that some sequence holds are written, nothing lies outside."""
    c = Cache([20, 20], 1, 16, 64, torch.bfloat16, gpu, width=2)
    k, v = rows_like("plain", 4, 1, 1, 64, torch.bfloat16, gpu)[1:]
    for bad in ([0, 4, 1], [0, 1, 900], [-5, 1, 2]):
        api.cache_append(k, v, c.kv[0], c.kv[1], c.table, ints([0, 0], gpu), ints(bad, gpu))
        torch.cuda.synchronize(gpu)
        assert api.device_status(gpu)[0] == 6, bad


def test_append_leaves_out_what_lies_outside(gpu):
    c = Cache([20, 20, 20], 2, 16, 64, torch.bfloat16, gpu, width=2)
    k, v = rows_like("plain", 6, 1, 2, 64, torch.bfloat16, gpu)[1:]
    before = c.kv.clone()
    c.table[1, 1] = 4000
    for start, rows in (([31, 31, 40], None), ([5, -1, 30], [0, -2, 1, 9, 6, 2])):
        c.kv.copy_(before)
        api.cache_append(k, v, c.kv[0], c.kv[1], c.table, ints(start, gpu), ints([0, 2, 4, 6], gpu),
                         rows=None if rows is None else ints(rows, gpu))
        torch.cuda.synchronize(gpu)
        assert api.device_status(gpu)[0] == 6
        want = before.clone()
        for b in range(3):
            for i in range(2):
                pos, row = start[b] + i, 2 * b + i if rows is None else rows[2 * b + i]
                if 0 <= pos < 32 and 0 <= row < 6 and 0 <= int(c.table[b, pos // 16]) < c.kv.shape[1]:
                    want[0, c.table[b, pos // 16], :, pos % 16] = k[row]
                    want[1, c.table[b, pos // 16], :, pos % 16] = v[row]
        assert torch.equal(c.kv.nan_to_num(77.0), want.nan_to_num(77.0))


# ------------------------------------------------------------------------------------------------ slots and pages
def pool_state(r, slots, width, page, pages, share):
    """Random slots; some share the full pages at their start."""
    free = r.sample(range(pages), pages)
    table, lens = [], []
    for s in range(slots):
        n = r.choice([0, 1, page - 1, page, page + 1, r.randrange(0, width * page + 1), r.randrange(0, width * page + 1)])
        n = min(n, width * page)
        row = []
        if s and share and r.random() < 0.5:
            o = r.randrange(s)
            row = table[o][: min(lens[o], n) // page]
        while len(row) < -(-n // page) and free:
            row = row + [free.pop()]
        n = min(n, len(row) * page)
        table.append(row + [r.choice([-1, 5, 1 << 29])] * (width - len(row)))
        lens.append(n)
    return table, lens


def check_update(gpu, kv, table, lens, src, new, page):
    want_kv = kv.clone()
    wt, wl, wi = ref.update(want_kv, table, lens, src, new, page)
    t, n = ints(table, gpu), ints(lens, gpu)
    info = api.cache_update(kv, t, n, ints(src, gpu), ints(new, gpu))
    ok(gpu)
    assert info.tolist() == wi
    assert t.tolist() == wt and n.tolist() == wl
    assert torch.equal(kv, want_kv)
    return wt, wl, wi


@pytest.mark.parametrize("seed", range(24))
def test_update_fuzz(gpu, seed):
    r = random.Random(seed)
    page, width, slots = r.choice([16, 32]), r.choice([1, 2, 7, 300]), r.choice([1, 2, 9, 70])
    planes, H, d = r.choice([1, 2, 6]), r.choice([1, 3]), r.choice([64, 128])
    pages = max(1, int(slots * width * r.choice([0.2, 0.6, 1.1])))
    kv = normal(planes, pages, H, page, d, dtype=DTYPES[seed % 2], device=gpu, seed=seed)
    table, lens = pool_state(r, slots, width, page, pages, share=seed % 3 > 0)
    for _ in range(3):
        src = [s if r.random() < 0.4 else r.randrange(slots) for s in range(slots)]
        new = [min(width * page, r.choice([0, lens[src[s]], lens[src[s]] + 1, r.randrange(width * page + 1),
                                           max(0, lens[src[s]] - r.randrange(20))])) for s in range(slots)]
        table, lens, _ = check_update(gpu, kv, table, lens, src, new, page)


def test_update_cases_by_hand(gpu):
    page, d = 16, 64
    kv = normal(2, 12, 1, page, d, dtype=torch.bfloat16, device=gpu)
    table, lens = [[3, 7, -1], [5, -1, -1], [-1, -1, -1]], [20, 16, 0]
    # fork slot 0 onto slot 2 while slot 0 is cut inside the page that slot 2 keeps whole: slot 0 gets its own copy
    t, n, info = check_update(gpu, kv, table, lens, [0, 1, 0], [10, 16, 17], page)
    assert t[2][0] == 3 and t[0][0] not in (3, 5, 7) and info == [2, 9]
    # every beam takes beam 0, one token more
    t, n, info = check_update(gpu, kv, t, n, [2, 2, 2], [18, 18, 18], page)
    assert t[0][0] == t[1][0] == t[2][0] == 3 and len({t[s][1] for s in range(3)}) == 3
    # all freed, then more than there are pages: nothing changes
    t, n, info = check_update(gpu, kv, t, n, [0, 1, 2], [0, 0, 0], page)
    assert info == [0, 8] and t == [[-1] * 3] * 3
    t2, n2, info = check_update(gpu, kv, t, n, [0, 1, 2], [48, 48, 48], page)
    assert info == [9, 12] and n2 == [48, 48, 48]
    t3, n3, info = check_update(gpu, kv[:, :8].contiguous(), t, n, [0, 1, 2], [48, 48, 48], page)
    assert info == [9, 8] and n3 == [0, 0, 0]


def test_update_many_pages(gpu):
    """A pool whose pages and tables take many rounds of the plan."""
    r = random.Random(1)
    page, width, slots, pages = 16, 900, 130, 70001
    kv = normal(1, pages, 1, page, 64, dtype=torch.bfloat16, device=gpu)
    table, lens = pool_state(r, slots, width, page, pages, share=True)
    src = [r.randrange(slots) for _ in range(slots)]
    new = [min(width * page, lens[s] + r.randrange(40)) for s in src]
    table, lens, _ = check_update(gpu, kv, table, lens, src, new, page)
    want = kv.clone()
    wt, wi = ref.compact(want, table, lens, page)
    t = ints(table, gpu)
    info = api.cache_compact(kv, t, ints(lens, gpu))
    ok(gpu)
    assert info.tolist() == wi and t.tolist() == wt and torch.equal(kv, want)


@pytest.mark.parametrize("seed", range(16))
def test_compact_fuzz(gpu, seed):
    r = random.Random(seed + 100)
    page, width, slots = r.choice([16, 64, 256]), r.choice([1, 3, 40]), r.choice([1, 3, 33])
    planes, H, d = r.choice([1, 2, 5]), r.choice([1, 2]), r.choice([64, 128])
    pages = max(1, int(slots * width * r.choice([0.5, 1.0, 2.0])))
    kv = normal(planes, pages, H, page, d, dtype=DTYPES[seed % 2], device=gpu, seed=seed)
    table, lens = pool_state(r, slots, width, page, pages, share=seed % 2 > 0)
    want = kv.clone()
    wt, wi = ref.compact(want, table, lens, page)
    t, n = ints(table, gpu), ints(lens, gpu)
    info = api.cache_compact(kv, t, n)
    ok(gpu)
    assert info.tolist() == wi and t.tolist() == wt and n.tolist() == lens and torch.equal(kv, want)
    assert api.cache_compact(kv, t, n).tolist() == [wi[0], 0], "a second pass has nothing to move"
    assert t.tolist() == wt and torch.equal(kv, want)


def test_pool_bad_device_values(gpu):
    """Recorded, info -1, and nothing changes."""
    page = 16
    kv = normal(2, 6, 1, page, 64, dtype=torch.bfloat16, device=gpu)
    good = ([[0, 1], [2, -1]], [20, 16], [0, 1], [20, 16])
    bad = [([[0, 6], [2, -1]], *good[1:]), ([[0, -1], [2, -1]], *good[1:]), (good[0], [33, 16], *good[2:]),
           (good[0], [-1, 16], *good[2:]), (*good[:2], [0, 2], good[3]), (*good[:2], [-1, 1], good[3]),
           (*good[:3], [20, 33]), (*good[:3], [20, -1])]
    before = kv.clone()
    for i, (table, lens, src, new) in enumerate(bad):
        t, n = ints(table, gpu), ints(lens, gpu)
        assert api.cache_update(kv, t, n, ints(src, gpu), ints(new, gpu)).tolist() == [-1, -1]
        assert api.device_status(gpu)[0] == 6
        assert t.tolist() == table and n.tolist() == lens and torch.equal(kv, before)
        if i < 4:
            assert api.cache_compact(kv, t, n).tolist() == [-1, -1]
            assert api.device_status(gpu)[0] == 6
            assert t.tolist() == table and torch.equal(kv, before)
    check_update(gpu, kv, *good, page)


# ------------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_serving_run(gpu, d, dtype):
    """Prompts, a fork, drafted trees with some nodes accepted, a slot freed, the pool compacted, one more token:
    after every step the cache holds what a plain list of rows holds, and attention over it agrees."""
    Hq, Hkv, page, slots, width, layers = 8, 2, 16, 4, 24, 2
    r = random.Random(7)
    kv = torch.full((2 * layers, 60, Hkv, page, d), float("nan"), dtype=dtype, device=gpu)
    table = torch.full((slots, width), -1, dtype=torch.int32, device=gpu)
    lens = torch.zeros(slots, dtype=torch.int32, device=gpu)
    held = [[torch.zeros((2, 0, Hkv, d), dtype=dtype, device=gpu) for _ in range(slots)] for _ in range(layers)]
    plain = list(range(slots))

    def update(src, new):
        info = api.cache_update(kv, table, lens, ints(src, gpu), ints(new, gpu)).tolist()
        assert 0 <= info[0] <= info[1]

    def step(nodes, accepted, seed, tree):
        """One step of every layer: nodes[s] tokens a slot, of which accepted[s] (indices) stay."""
        T = sum(nodes)
        cu = ints(ref.offsets(nodes), gpu)
        start = lens.clone()
        mask, bits = None, None
        if tree:
            words, bits, parents = masks_of("tree", nodes, seed)
            mask = api.tree_mask(ints(parents, gpu), cu, words)
        new = []
        for layer in range(layers):
            q, k, v = rows_like("fused", T, Hq, Hkv, d, dtype, gpu, seed=seed + layer)
            kc, vc = kv[2 * layer], kv[2 * layer + 1]
            if int(start.sum()) == 0:
                o, lse = api.forward_prompt(q, k, v, cu)
            else:
                o, lse = api.forward_tree(q, k, v, kc, vc, table, start, cu, mask=mask)
            want = ref.forward(q, k, v, nodes, d ** -0.5, ctx=lambda b: held[layer][b],
                               seen_nodes=None if bits is None else (lambda b, n: bits[b]))
            ref.assert_close(o, lse, want, T)
            new.append((k, v))
        update(plain, [int(n) + len(a) for n, a in zip(start, accepted)])
        at = ref.offsets(nodes)
        rows = [at[s] + i for s in range(slots) for i in accepted[s]]
        cu_kept = ints(ref.offsets([len(a) for a in accepted]), gpu)
        for layer, (k, v) in enumerate(new):
            api.cache_append(k, v, kv[2 * layer], kv[2 * layer + 1], table, start, cu_kept, rows=ints(rows, gpu))
            for s in range(slots):
                pick = torch.tensor([at[s] + i for i in accepted[s]], dtype=torch.long, device=gpu)
                held[layer][s] = torch.cat([held[layer][s], torch.stack([k[pick], v[pick]])], 1)
        ok(gpu)
        for layer in range(layers):
            for s in range(slots):
                got = torch.stack([ref.rows_of_cache(kv[2 * layer + i], table, s, int(lens[s])) for i in range(2)])
                assert torch.equal(got, held[layer][s])

    prompts = [100, 37, 0, 16]
    step(prompts, [list(range(n)) for n in prompts], 10, False)
    update([0, 1, 0, 3], [100, 37, 100, 16])  # slot 2 forks slot 0
    for layer in range(layers):
        held[layer][2] = held[layer][0].clone()
    nodes = [12, 5, 9, 0]
    step(nodes, [sorted(r.sample(range(n), n // 2)) for n in nodes], 20, True)
    update([0, 0, 2, 3], [0, 60, int(lens[2]), 0])  # 0 and 3 freed, 1 becomes the start of 0
    for layer in range(layers):
        held[layer][1] = held[layer][0][:, :60]
        held[layer][0] = held[layer][0][:, :0]
        held[layer][3] = held[layer][3][:, :0]
    used = len({p for s in range(slots) for p in table[s, : -(-int(lens[s]) // page)].tolist()})
    info = api.cache_compact(kv, table, lens).tolist()
    assert info[0] == used and int(table.max()) < used
    step([0, 1, 1, 0], [[], [0], [0], []], 30, False)
