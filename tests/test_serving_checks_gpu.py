"""The serving operators in the library's test builds, and what their wrappers refuse.

In the bounds-checked build nothing fires on valid inputs and the results are right. In the build
that leaves out a copy in every CTA the attention kernel reports FA_ERR_TIMEOUT, stops cleanly and
leaves the context usable.
"""

import math

import pytest
import torch

import serving_ref as ref
from io_aware_exact_04_gb300 import _lib, api
from test_serving_gpu import Cache, ints, masks_of, normal, ok, rows_like

pytestmark = pytest.mark.gpu


@pytest.fixture
def build(gpu, monkeypatch):
    def use(name):
        lib = _lib.load(name)
        monkeypatch.setattr(api, "_lib_fa", lambda: lib)
        api.device_status(gpu)
    return use


@pytest.mark.parametrize("d", [64, 128])
def test_debug_build_is_silent_and_right(build, gpu, d):
    build("libfa_debug.so")
    for lens, Hq, Hkv in (([300, 1, 0, 129], 6, 2), ([700], 2, 2)):
        T = sum(lens)
        q, k, v = rows_like("fused", T, Hq, Hkv, d, torch.bfloat16, gpu)
        o, lse = api.forward_prompt(q, k, v, ints(ref.offsets(lens), gpu))
        ok(gpu)
        ref.assert_close(o, lse, ref.forward(q, k, v, lens, d ** -0.5), T)
    lens, nodes, Hq, Hkv = [2000, 77, 513], [40, 1, 64], 8, 2
    words, bits, parents = masks_of("tree", nodes)
    T = sum(nodes)
    q, k, v = rows_like("plain", T, Hq, Hkv, d, torch.float16, gpu)
    c = Cache(lens, Hkv, 32, d, torch.float16, gpu)
    cu = ints(ref.offsets(nodes), gpu)
    mask = api.tree_mask(ints(parents, gpu), cu, words)
    o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu, mask=mask)
    ok(gpu)
    ref.assert_close(o, lse, ref.forward(q, k, v, nodes, d ** -0.5, ctx=c.ctx, seen_nodes=lambda b, n: bits[b][:, :n]), T)
    api.cache_append(k, v, c.kv[0], c.kv[1], c.table, ints([0, 0, 0], gpu), cu)
    ok(gpu)
    kv = normal(2, 30, 1, 16, d, dtype=torch.bfloat16, device=gpu)
    table, n = ints([[3, 9, -1], [20, 21, 22]], gpu), ints([30, 48], gpu)
    assert api.cache_update(kv, table, n, ints([1, 1], gpu), ints([20, 48], gpu)).tolist() == [1, 25]
    assert api.cache_compact(kv, table, n).tolist() == [4, 3]  # pages 20, 21, 22 and the first free one, 0
    ok(gpu)


@pytest.mark.parametrize("d", [64, 128])
def test_a_copy_that_never_arrives(build, gpu, d):
    c = Cache([4000], 1, 64, d, torch.bfloat16, gpu)
    q, k, v = rows_like("plain", 1, 4, 1, d, torch.bfloat16, gpu)
    cu = ints([0, 1], gpu)
    P = 700
    pq, pk, pv = rows_like("plain", P, 2, 1, d, torch.bfloat16, gpu)
    pcu = ints([0, P], gpu)
    build("libfa_withhold.so")
    for call in (lambda: api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu),
                 lambda: api.forward_prompt(pq, pk, pv, pcu)):
        call()
        torch.cuda.synchronize(gpu)
        code, detail = api.device_status(gpu)
        assert code == 5 and 60 <= detail[1] <= 80, detail
    build("libfa.so")
    o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu)
    ok(gpu)
    ref.assert_close(o, lse, ref.forward(q, k, v, [1], d ** -0.5, ctx=c.ctx), 1)
    o, lse = api.forward_prompt(pq, pk, pv, pcu)
    ok(gpu)
    ref.assert_close(o, lse, ref.forward(pq, pk, pv, [P], d ** -0.5), P)


def test_wrappers_refuse(gpu):
    T, Hq, Hkv, d, page = 6, 4, 2, 64, 16
    q, k, v = rows_like("plain", T, Hq, Hkv, d, torch.bfloat16, gpu)
    c = Cache([20, 20], Hkv, page, d, torch.bfloat16, gpu)
    cu = ints([0, 3, 6], gpu)
    mask = torch.zeros((T, 1), dtype=torch.int32, device=gpu)
    base = dict(q=q, k=k, v=v, k_cache=c.kv[0], v_cache=c.kv[1], table=c.table, lens=c.lens, cu_nodes=cu, mask=mask)

    def bad(fn, args, **kw):
        with pytest.raises(ValueError):
            fn(**{**args, **kw})

    odd = torch.zeros((T, Hq, d + 1), dtype=torch.bfloat16, device=gpu)[..., :d]  # rows not a multiple of 8 apart
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(q=q.cpu()), dict(q=odd), dict(q=q[:, :3]), dict(q=q[:1].expand(T, -1, -1)),
               dict(q=q.transpose(1, 2)), dict(k=k.half()), dict(k=k[:5]), dict(v=v[:, :1]), dict(v=v.cpu()),
               dict(k_cache=c.kv[0][:, :1]), dict(k_cache=c.kv[0].half()), dict(v_cache=c.kv[1][1:]),
               dict(v_cache=c.kv[1].cpu()), dict(table=c.table.long()), dict(table=c.table[:1]), dict(table=c.table[:, :0]),
               dict(table=c.table.t()), dict(lens=c.lens.long()), dict(lens=c.lens[:1]), dict(cu_nodes=cu.long()),
               dict(cu_nodes=cu[:0]), dict(cu_nodes=cu[None]), dict(mask=mask[:5]), dict(mask=mask.long()),
               dict(mask=mask[:, :0]), dict(mask=mask[:, 0]), dict(out=torch.empty_like(q)[:5]),
               dict(lse=torch.empty((Hq, T + 1), device=gpu)), dict(lse=torch.empty((T, Hq), device=gpu).t()),
               dict(workspace=torch.empty(100, device=gpu))):
        bad(api.forward_tree, base, **kw)
    with pytest.raises(_lib.FaError):  # a workspace that is too small
        api.forward_tree(**base, workspace=torch.empty(256, dtype=torch.uint8, device=gpu))
    with pytest.raises(_lib.FaError):  # a page size that is not served
        api.forward_tree(**{**base, "k_cache": c.kv[0][:, :, :8], "v_cache": c.kv[1][:, :, :8]})
    with pytest.raises(_lib.FaError):
        api.forward_prompt(q, k, v, cu, scale=0.0)
    z = torch.zeros((T, 4, 32), dtype=torch.bfloat16, device=gpu)
    with pytest.raises(_lib.FaError):
        api.forward_prompt(z, z, z, cu)
    ap = dict(k=k, v=v, k_cache=c.kv[0], v_cache=c.kv[1], table=c.table, start=c.lens, cu=cu)
    for kw in (dict(k=k.float()), dict(v=v[:3]), dict(start=c.lens[:1]), dict(cu=cu.cpu()), dict(rows=cu.long()),
               dict(rows=cu[None]), dict(k_cache=c.kv[0].transpose(2, 3)), dict(table=c.table[:1])):
        bad(api.cache_append, ap, **kw)
    kv = normal(4, 10, Hkv, page, d, dtype=torch.bfloat16, device=gpu)
    up = dict(kv=kv, table=c.table, lens=c.lens, src=ints([0, 1], gpu), new_lens=c.lens)
    for kw in (dict(kv=kv[0]), dict(kv=kv.float()), dict(kv=kv.transpose(2, 3)), dict(kv=kv[:, :, :1]), dict(kv=kv[:0]),
               dict(kv=kv[:1].expand(4, -1, -1, -1, -1)), dict(table=c.table[:, 1:]), dict(table=c.table.long()),
               dict(lens=c.lens[:1]), dict(src=ints([0], gpu)), dict(src=cu), dict(new_lens=c.lens.long()),
               dict(workspace=torch.empty(100, device=gpu))):
        bad(api.cache_update, up, **kw)
    with pytest.raises(_lib.FaError):
        api.cache_update(**up, workspace=torch.empty(256, dtype=torch.uint8, device=gpu))
    ok(gpu)


def test_empty_calls(gpu):
    """No tokens, no sequences: nothing is launched and nothing fails."""
    d = 64
    c = Cache([20], 2, 16, d, torch.bfloat16, gpu)
    none = torch.empty((0, 2, d), dtype=torch.bfloat16, device=gpu)
    for cu in (ints([0], gpu), ints([0, 0], gpu)):
        o, lse = api.forward_prompt(none, none, none, cu)
        assert o.shape == (0, 2, d) and lse.shape == (2, 0)
        B = cu.numel() - 1
        o, lse = api.forward_tree(none, none, none, c.kv[0], c.kv[1], c.table, c.lens[:B], cu)
        assert o.shape == (0, 2, d)
        api.cache_append(none, none, c.kv[0], c.kv[1], c.table, c.lens[:B], cu)
    assert api.tree_mask(ints([], gpu), ints([0], gpu), 1).shape == (0, 1)
    # tokens of no sequence: all rows stay
    x = normal(3, 2, d, dtype=torch.bfloat16, device=gpu)
    out = torch.full_like(x, 2.0)
    api.forward_prompt(x, x, x, ints([0], gpu), out=out)
    api.forward_prompt(x, x, x, ints([0, 0, 0], gpu), out=out)
    api.forward_tree(x, x, x, c.kv[0], c.kv[1], c.table, c.lens, ints([0, 0], gpu), out=out)
    ok(gpu)
    assert (out == 2.0).all()


@pytest.mark.parametrize("seed", range(12))
def test_tree_fuzz(gpu, seed):
    """Random batches over the whole range of layouts; every second one poisoned workspaces."""
    import random
    r = random.Random(seed)
    d, dtype = r.choice([64, 128]), r.choice([torch.bfloat16, torch.float16])
    Hkv = r.choice([1, 2, 3])
    Hq = Hkv * r.choice([1, 2, 3, 4, 6, 9])
    B = r.choice([1, 3, 9, 33])
    page = r.choice([16, 32, 64, 128, 256])
    lens = [r.choice([0, 1, 127, 128, 129, r.randrange(700), r.randrange(3000 // B + 2)]) for _ in range(B)]
    nodes = [r.choice([0, 1, 1, 2, r.randrange(1, 70), r.randrange(1, 200) if B < 9 else 5]) for _ in range(B)]
    nodes[0] = max(1, nodes[0])
    T = sum(nodes)
    kind = r.choice([None, "tree", "random"])
    q, k, v = rows_like(r.choice(["plain", "fused", "heads"]), T, Hq, Hkv, d, dtype, gpu, seed=seed)
    c = Cache(lens, Hkv, page, d, dtype, gpu, seed=seed, order=r.choice(["hpd", "phd"]))
    cu, mask, seen = ints(ref.offsets(nodes), gpu), None, None
    if kind:
        words, bits, _ = masks_of(kind, nodes, seed)
        mask = torch.cat([ref.pack_bits(s, words) for s in bits]).to(gpu)
        seen = lambda b, n: bits[b][:, :n]  # noqa: E731
    ws = torch.full((api._tree_workspace(gpu.index, d),), 0xFF if seed % 2 else 0, dtype=torch.uint8, device=gpu)
    o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu, mask=mask, workspace=ws)
    ok(gpu)
    ref.assert_close(o, lse, ref.forward(q, k, v, nodes, 1 / math.sqrt(d), ctx=c.ctx, seen_nodes=seen), T)
    p, lse = api.forward_prompt(q, k, v, cu)
    ok(gpu)
    ref.assert_close(p, lse, ref.forward(q, k, v, nodes, 1 / math.sqrt(d)), T)


def test_many_repetitions_agree(gpu):
    """A thousand calls with poisoned outputs and workspaces, bit for bit the same."""
    for d, lens, nodes in ((128, [900, 130, 2500, 64], [9, 33, 1, 70]), (64, [900, 130, 2500, 64], [9, 140, 1, 70])):
        T = sum(nodes)
        q, k, v = rows_like("plain", T, 8, 2, d, torch.bfloat16, gpu)
        c = Cache(lens, 2, 32, d, torch.bfloat16, gpu)
        cu = ints(ref.offsets(nodes), gpu)
        ws = torch.empty(api._tree_workspace(gpu.index, d), dtype=torch.uint8, device=gpu)
        first = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu)
        prompt = api.forward_prompt(q, k, v, cu)
        bad = torch.zeros((), dtype=torch.int64, device=gpu)
        for _ in range(500):
            ws.fill_(0xFF)
            out = torch.full_like(q, float("nan"))
            o, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu, out=out, workspace=ws)
            bad += (o != first[0]).any().long() + (lse != first[1]).any().long()
            o, lse = api.forward_prompt(q, k, v, cu, out=torch.full_like(q, float("nan")))
            bad += (o != prompt[0]).any().long() + (lse != prompt[1]).any().long()
        ok(gpu)
        assert int(bad) == 0
