"""Attention over a cache in 8 bits: the library's test builds, invalid values on the device, what a NaN reaches,
scales far apart, memory far away, other streams, graphs, and a serving loop of all the operators together.

FEW and SOME have few rows a sequence (decoding, small drafts), up to 8 and up to 32, MANY many: different kernels.
"""

import math

import pytest
import torch

from io_aware_exact_04_gb300 import _lib, api
from tests import cache8_ref as ref
from tests import serving_ref
from tests.test_tree8_gpu import BF16, E4M3, FP16, Made, ints

pytestmark = pytest.mark.gpu
FEW = dict(lens=[300, 0, 1000, 64], nodes=[2, 1, 1, 3], Hq=4, H=2)
SOME = dict(lens=[300, 0, 1000, 64], nodes=[6, 5, 4, 7], Hq=8, H=2)
MANY = dict(lens=[300, 0, 700, 64], nodes=[20, 9, 40, 33], Hq=8, H=2)
BOTH = pytest.mark.parametrize("shape", [FEW, SOME, MANY], ids=["few", "some", "many"])
TYPES = pytest.mark.parametrize("dtype", [BF16, FP16])


def made(gpu, shape, d=128, page=32, block=16, dtype=BF16, **kw):
    return Made(gpu, shape["lens"], shape["nodes"], shape["Hq"], shape["H"], d, page, block, dtype, **kw)


def rows_of(m, b):
    at = serving_ref.offsets(m.nodes)
    return slice(at[b], at[b + 1])


@pytest.fixture
def build(gpu, monkeypatch):
    def use(name):
        lib = _lib.load(name)
        monkeypatch.setattr(api, "_lib_fa", lambda: lib)
        api.device_status(gpu)
    return use


@pytest.mark.parametrize("d", [64, 128])
@BOTH
def test_debug_build_is_silent_and_right(build, gpu, shape, d):
    build("libfa_debug.so")
    for dtype in (BF16, FP16):
        for tree in (False, True):
            made(gpu, shape, d=d, dtype=dtype, tree=tree).check()


@pytest.mark.parametrize("nodes,Hq", [(1, 4), (4, 4), (40, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_copy_that_never_arrives(build, gpu, d, nodes, Hq):
    """The wait for it runs out, the kernel says where and stops; the same call of the library's own build is right after."""
    m = Made(gpu, [4000], [nodes], Hq, 1, d, 64, 32, BF16)
    build("libfa_withhold.so")
    m.call()
    torch.cuda.synchronize(gpu)
    code, detail = api.device_status(gpu)
    assert code == 5 and 60 <= detail[1] <= 99, detail
    build("libfa.so")
    m.check()


@BOTH
@TYPES
def test_rows_behind_the_last_sequence_stay(gpu, shape, dtype):
    m = made(gpu, shape, dtype=dtype, tail=7)
    out = torch.full_like(m.q, 3.0)
    lse = torch.full((m.q.shape[1], m.q.shape[0]), 3.0, device=gpu)
    m.check(m.call(out=out, lse=lse))
    assert bool((out[m.T:] == 3.0).all()) and bool((lse[:, m.T:] == 3.0).all())
    o, none = m.call(lse=False)
    assert torch.equal(o[: m.T], out[: m.T])


@BOTH
def test_strides_and_alignment(gpu, shape):
    """Rows inside a wider tensor, heads before tokens, pages with tokens before heads, and scales of both planes in
    one tensor: the same bits."""
    m = made(gpu, shape, tail=0)
    want = m.call()
    q, k, v, kc, vc, ks, vs = m.q, m.k, m.v, m.kc, m.vc, m.ks, m.vs
    T, d = q.shape[0], q.shape[2]
    wide = torch.full((T, q.shape[1] + 2 * k.shape[1] + 1, d), math.nan, dtype=q.dtype, device=gpu)
    at = 0
    for name in ("q", "k", "v"):
        x = getattr(m, name)
        wide[:, at:at + x.shape[1]] = x
        setattr(m, name, wide[:, at:at + x.shape[1]])
        at += x.shape[1]
    other = [c.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(E4M3) for c in (kc, vc)]
    m.kc, m.vc = other
    both = torch.stack([ks, vs], 1)
    m.ks, m.vs = both[:, 0], both[:, 1]
    for out in (None, torch.empty((q.shape[1], T, d), dtype=q.dtype, device=gpu).transpose(0, 1)):
        got = m.call(out=out)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert api.device_status(gpu)[0] == 0


@BOTH
@TYPES
def test_invalid_values_on_the_device(gpu, shape, dtype):
    """A page id outside the cache counts as zeros, lengths and offsets are taken into their ranges; each is recorded
    with code 6, and no other sequence is concerned."""
    m = made(gpu, shape, dtype=dtype)
    want = m.call()
    assert api.device_status(gpu)[0] == 0
    for bad in (-1, m.kc.shape[0], 1 << 30, -(1 << 31)):
        m.table[0, 1] = bad  # tokens 32 .. 63 of sequence 0
        got = m.call()
        code, _ = api.device_status(gpu)
        assert code == 6
        assert torch.equal(got[0][rows_of(m, 2)], want[0][rows_of(m, 2)])
    page = m.table_list[0][1]
    bytes_of = [c.view(torch.uint8)[page] for c in (m.kc, m.vc)]
    was = [x.clone() for x in bytes_of]
    m.table[0, 1] = page
    for x in bytes_of:
        x.zero_()
    # (within the bounds: a page that is there brings its scales, and with them another reference for those of V)
    m.check(got)
    for x, y in zip(bytes_of, was):
        x.copy_(y)
    assert api.device_status(gpu)[0] == 0
    m.len_t[1] = -5  # as 0, which it is
    got = m.call()
    assert api.device_status(gpu)[0] == 6 and torch.equal(got[0][: m.T], want[0][: m.T])
    m.len_t[1] = 0
    # a length past the table: taken as all of it (the entries of this sequence's last pages are -1: zeros)
    m.len_t[2] = 1 << 29
    got = m.call()
    assert api.device_status(gpu)[0] == 6
    for b in (0, 1, 3):
        assert torch.equal(got[0][rows_of(m, b)], want[0][rows_of(m, b)])
    m.len_t[2] = m.lens[2]
    # an offset past the rows: the last sequence ends with them; one that falls: a sequence without tokens
    m.cu[4] = m.q.shape[0] + 100
    m.call()
    assert api.device_status(gpu)[0] == 6
    m.cu[4] = m.cu[3] - 1
    got = m.call()
    assert api.device_status(gpu)[0] == 6
    for b in range(3):
        assert torch.equal(got[0][rows_of(m, b)], want[0][rows_of(m, b)])
    m.cu[4] = m.T
    m.check()


@BOTH
@TYPES
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_what_a_nan_reaches(gpu, shape, dtype, bad):
    """A query: its own row. K of a node: the rows that see it. V of a node, K and V in the cache: rows of its sequence
    and key/value head only."""
    m = made(gpu, shape, dtype=dtype, tail=0)
    G = shape["Hq"] // shape["H"]
    o, lse = m.call()
    at = serving_ref.offsets(m.nodes)

    def changed():
        got, glse = m.call()
        assert api.device_status(gpu)[0] == 0
        rows = (got.view(torch.int16) != o.view(torch.int16)).any(-1) | (glse.t() != lse.t())
        return got, glse, rows  # [T, Hq]; NaN != anything

    q, k, v = m.q, m.k, m.v
    for b in (0, 2, 3):
        for i in {0, m.nodes[b] - 1}:
            t = at[b] + i
            m.q = q.clone()
            m.q[t, 1, 5] = bad
            got, glse, rows = changed()
            expect = torch.zeros_like(rows)
            expect[t, 1] = True
            assert torch.equal(rows, expect) and bool(got[t, 1].isnan().all()) and bool(glse[1, t].isnan())
            m.q, m.k = q, k.clone()
            m.k[t, 0] = math.nan  # (of an infinity the sign of a score decides)
            got, glse, rows = changed()
            expect = torch.zeros_like(rows)
            expect[t:at[b + 1], :G] = True
            assert torch.equal(rows, expect) and bool(got[t:at[b + 1], :G].isnan().all())
            m.k, m.v = k, v.clone()
            m.v[t, 1, 3] = bad
            got, glse, rows = changed()
            assert not bool(rows[:, :G].any()) and not bool(rows[:at[b]].any()) and not bool(rows[at[b + 1]:].any())
            assert torch.equal(glse, lse)
            assert not bool(got[t:at[b + 1], G:, 3].isfinite().any())
            m.v = v
    for b, place in ((0, 0), (0, 299), (2, 130)):
        page = m.table_list[b][place // m.page]
        for c in (m.kc, m.vc):
            x = c.view(torch.uint8)[page, 1, place % m.page]
            was = x[7].clone()
            x[7] = 0x7F
            got, glse, rows = changed()
            x[7] = was
            assert not bool(rows[:, :G].any()) and not bool(rows[:at[b]].any()) and not bool(rows[at[b + 1]:].any())
            hit = got[at[b]:at[b + 1], G:]
            assert bool((hit if c is m.kc else hit[..., 7]).isnan().all())
            assert torch.equal(glse, lse) if c is m.vc else bool(glse[G:, at[b]:at[b + 1]].isnan().all())
    m.check()


@BOTH
@TYPES
@pytest.mark.parametrize("d", [64, 128])
def test_scales_far_apart(gpu, shape, dtype, d):
    """Blocks of V whose scales lie 2^20 and more apart, in any order."""
    made(gpu, shape, d=d, dtype=dtype, spread=5.0, seed=4).check()


@BOTH
@TYPES
def test_small_probabilities_beside_a_large_one(gpu, shape, dtype):
    """A key that takes nearly all of a row and has no value of its own: what is left is the sum of probabilities of
    2^-18 and less, each rounded relative to itself."""
    m = made(gpu, shape, dtype=dtype, seed=5, tail=0, spread=0.0)
    lens = m.lens
    m.q.mul_(0.25)
    for b in (0, 2):
        page = m.table_list[b][0]
        for h in range(shape["H"]):
            # key 0 of the sequence along all its queries' common part
            m.q[rows_of(m, b), h * (shape["Hq"] // shape["H"]):(h + 1) * (shape["Hq"] // shape["H"]), :16] = 2.0
            m.kc.view(torch.uint8)[page, h, 0] = 0
            m.kc.view(torch.uint8)[page, h, 0, :16] = 0x7E  # 448
            m.ks[page, h, 0] = 2.0 ** -6 * (18 * math.log(2) / (16 * 2.0 * 7.0 * m.scale))
            m.vc.view(torch.uint8)[page, h, 0] = 0
    o, lse = m.check()
    assert lens[0] and float(o[rows_of(m, 0)].abs().max()) < 2.0 ** -5


def test_pages_far_apart(gpu):
    """Pages past 2^31 and 2^32 bytes: the same bits as nearby."""
    if torch.cuda.mem_get_info(gpu)[0] < 24 << 30:
        pytest.skip("needs 24 GB of free memory")
    H, page, d, far = 8, 64, 128, 70000
    pools = [torch.empty((far, H, page, d), dtype=torch.uint8, device=gpu) for _ in range(2)]
    scales = [torch.empty((far, H, 2), device=gpu) for _ in range(2)]
    for shape in (FEW, SOME, MANY):
        m = Made(gpu, shape["lens"], shape["nodes"], 16, H, d, page, 32, BF16, tail=0)
        want = m.check()
        n = m.kc.shape[0]
        places = torch.tensor([far - 1, 32767, 32768, 65535, 65536, 40000, 16384, 69000] + list(range(50000, 50000 + n)),
                              device=gpu)[:n]
        for to, s, c, of in zip(pools, scales, (m.kc, m.vc), (m.ks, m.vs)):
            to[places] = c.view(torch.uint8)
            s[places] = of
        table = torch.where(m.table >= 0, places[m.table.clamp(min=0).long()].int(), m.table)
        m.kc, m.vc = (p.view(E4M3) for p in pools)
        m.ks, m.vs = scales
        m.table = table.contiguous()
        got = m.call()
        assert api.device_status(gpu)[0] == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del m, got, want, table
    del pools, scales
    torch.cuda.empty_cache()


@BOTH
def test_another_stream(gpu, shape):
    m = made(gpu, shape)
    want = m.call()
    torch.cuda.synchronize(gpu)
    s = torch.cuda.Stream(gpu)
    with torch.cuda.stream(s):
        got = [m.call() for _ in range(3)]
    s.synchronize()
    for o, lse in got:
        assert torch.equal(o[: m.T], want[0][: m.T]) and torch.equal(lse[:, : m.T], want[1][:, : m.T])


def test_two_graphs_with_workspaces_of_their_own(gpu):
    """Captured at once, replayed at once on two streams, then with other lengths."""
    ms = [made(gpu, FEW, tail=0, seed=1), made(gpu, MANY, tail=0, seed=2)]
    need = api._tree_workspace(gpu.index, 128, "fa_forward_tree_8bit")
    spaces = [torch.empty(need, dtype=torch.uint8, device=gpu) for _ in ms]
    want = [m.check() for m in ms]
    graphs, outs = [], []
    for m, w in zip(ms, spaces):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(m.call(workspace=w))
        graphs.append(graph)
    streams = [torch.cuda.Stream(gpu) for _ in ms]
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize(gpu)
    for (o, lse), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)
    for m, graph, out in zip(ms, graphs, outs):
        m.lens = [n // 2 for n in m.lens]
        m.nodes = [m.nodes[0] + m.nodes[3], m.nodes[1], m.nodes[2], 0]
        m.len_t.copy_(ints(m.lens, gpu))
        m.cu.copy_(ints(serving_ref.offsets(m.nodes), gpu))
        graph.replay()
        m.check(out)


@TYPES
def test_a_serving_loop(gpu, dtype):
    """Prompts rotated and appended in two parts, a decoding step, drafted trees whose accepted path is appended, slots
    that fork, compaction, another step: the cache against its plain form, the attention against the definition over
    what the cache then holds."""
    H, Hq, d, page, block, width, slots = 2, 8, 64, 32, 16, 8, 3
    n_pages, scale = 40, d ** -0.5
    g = torch.Generator().manual_seed(9)
    pool = torch.zeros((2, n_pages, H, page, d)).to(E4M3).to(gpu)
    scales = torch.ones((2, n_pages, H, page // block), device=gpu)
    plain, plain_s = pool.cpu(), scales.cpu()
    table = torch.full((slots, width), -1, dtype=torch.int32)
    free = torch.randperm(n_pages, generator=g).tolist()
    lens = [0] * slots
    angles = api.rotary_angles(width * page, d, device=gpu)

    def rows(T):
        return [torch.randn((T, h, d), generator=g).to(dtype).to(gpu) for h in (Hq, H, H)]

    def room(n):  # pages for n[b] tokens more
        for b in range(slots):
            for j in range(width):
                if j * page < lens[b] + n[b] and table[b, j] < 0:
                    table[b, j] = free.pop()

    def compare():
        assert api.device_status(gpu)[0] == 0
        for b in range(slots):
            for j in range(-(-lens[b] // page)):
                p, n = int(table[b, j]), min(page, lens[b] - j * page)
                blocks = -(-n // block)
                assert torch.equal(scales[:, p, :, :blocks].cpu(), plain_s[:, p, :, :blocks])
                assert torch.equal(pool[:, p, :, :n].cpu().view(torch.uint8), plain[:, p, :, :n].view(torch.uint8))

    def attend(q, k, v, n, seen=None, mask=None):
        cu, at, tb = ints(serving_ref.offsets(n), gpu), ints(lens, gpu), table.to(gpu)
        got = api.forward_tree(q, k, v, pool[0], pool[1], tb, at, cu, mask=mask, k_scale=scales[0], v_scale=scales[1])
        whole = [ref.dequantised(pool[i], scales[i]) for i in range(2)]
        ctx = lambda b: [serving_ref.rows_of_cache(x, tb, b, lens[b]) for x in whole]  # noqa: E731
        serving_ref.assert_close(*got, serving_ref.forward(q, k, v, n, scale, ctx=ctx, seen_nodes=seen), sum(n))

    def extend(n):
        """New tokens rotated and appended, their attention over what was there before, as a chain."""
        T = sum(n)
        q, k, v = rows(T)
        room(n)
        cu, at, tb = ints(serving_ref.offsets(n), gpu), ints(lens, gpu), table.to(gpu)
        places = [lens[b] + i for b in range(slots) for i in range(n[b])]
        want = [ref.rotated(x, angles, places, False) for x in (q, k)]
        before = (pool.clone(), scales.clone())
        qr, kr = api.rotary_append(q, k, v, pool[0], pool[1], tb, at, cu, angles, k_scale=scales[0], v_scale=scales[1])
        for x, y in zip((qr, kr), want):
            assert torch.equal(x.cpu(), y.to(dtype))
        after = (pool.clone(), scales.clone())
        pool.copy_(before[0])
        scales.copy_(before[1])
        attend(qr, kr, v, n)  # over the tokens before
        pool.copy_(after[0])
        scales.copy_(after[1])
        ref.append(want[1], plain[0], plain_s[0], table.tolist(), lens, n)
        ref.append(v.float().cpu(), plain[1], plain_s[1], table.tolist(), lens, n)
        for b in range(slots):
            lens[b] += n[b]
        compare()

    extend([70, 33, 5])
    extend([40, 0, 27])
    extend([1, 1, 1])
    # drafted trees: rotated at their depth, looked at, and one path of each accepted
    parents = [[-1, 0, 0, 1, 1, 2], [-1], [-1, 0, 1, 1, 3]]
    n = [len(p) for p in parents]
    cu, T = ints(serving_ref.offsets(n), gpu), sum(n)
    q, k, v = rows(T)
    depth = lambda p, i: 0 if p[i] < 0 else 1 + depth(p, p[i])  # noqa: E731
    places = [lens[b] + depth(parents[b], i) for b in range(slots) for i in range(n[b])]
    qr, kr = api.rotary(q, k, angles, ints(places, gpu))
    assert torch.equal(kr.cpu(), ref.rotated(k, angles, places, False).to(dtype))
    mask = api.tree_mask(ints(sum(parents, []), gpu), cu, 1)
    see = [serving_ref.ancestors(p).to(gpu) for p in parents]
    attend(qr, kr, v, n, seen=lambda b, m: see[b], mask=mask)
    paths = [[0, 1, 4], [0], [0, 1, 3, 4]]
    at0 = serving_ref.offsets(n)
    take = [at0[b] + i for b in range(slots) for i in paths[b]]
    m = [len(p) for p in paths]
    room(m)
    api.cache_append(kr, v, pool[0], pool[1], table.to(gpu), ints(lens, gpu), ints(serving_ref.offsets(m), gpu), rows=ints(take, gpu),
                     k_scale=scales[0], v_scale=scales[1])
    for i, x in enumerate((kr, v)):
        ref.append(x.float().cpu(), plain[i], plain_s[i], table.tolist(), lens, m, rows=take)
    for b in range(slots):
        lens[b] += m[b]
    compare()
    # slot 1 becomes a copy of slot 0, slot 2 loses its last tokens
    td, ld = table.to(gpu), ints(lens, gpu)
    keep = [lens[0], lens[0], lens[2] - 6]
    info = api.cache_update(pool, td, ld, ints([0, 0, 2], gpu), ints(keep, gpu), scales=scales)
    new, new_lens, want_info = serving_ref.update(plain.view(torch.uint8), table.tolist(), lens, [0, 0, 2], keep, page)
    assert info.tolist() == want_info and td.tolist() == new and ld.tolist() == new_lens
    part = keep[1] % page
    if part:
        to, of = new[1][keep[1] // page], int(table[0, keep[1] // page])
        if to != of:
            plain_s[:, to, :, : -(-part // block)] = plain_s[:, of, :, : -(-part // block)]
    table, lens = td.cpu(), list(keep)
    compare()
    api.cache_compact(pool, td, ld, scales=scales)
    moved = td.cpu()
    old, old_s = plain.clone(), plain_s.clone()
    for b in range(slots):
        for j in range(-(-lens[b] // page)):
            plain[:, int(moved[b, j])], plain_s[:, int(moved[b, j])] = old[:, int(table[b, j])], old_s[:, int(table[b, j])]
    used = {int(moved[b, j]) for b in range(slots) for j in range(-(-lens[b] // page))}
    assert used == set(range(len(used)))
    table = moved
    free = [x for x in range(n_pages) if x not in used]
    for b in range(slots):
        table[b, -(-lens[b] // page):] = -1
    compare()
    extend([1, 2, 3])


@TYPES
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("nodes,Hq,H", [([1] * 20 + [30, 0, 2], 1, 1), ([1, 1, 40] + [1] * 30, 4, 2), ([2] * 9 + [70], 6, 2)])
def test_one_sequence_with_many_rows_among_few(gpu, dtype, nodes, Hq, H, tree):
    """The average decides which kernel runs: a sequence with many more rows is several items."""
    lens = [(137 * i) % 900 for i in range(len(nodes))]
    for d in (64, 128):
        Made(gpu, lens, nodes, Hq, H, d, 32, 16, dtype, seed=8, tree=tree).check()
