"""Rotation and the way into the cache, of 16 bits and of 8, against plain forms."""

import math

import pytest
import torch

from io_aware_exact_04_gb300 import api
from tests import cache8_ref as ref

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def ints(x, gpu):
    return torch.tensor(x, dtype=torch.int32, device=gpu)


def strided(x, how):
    """The same values with other strides: a view of a wider projection, or heads outside tokens."""
    if how == "wide":
        t, h, d = x.shape
        y = torch.empty((t, h + 3, d + 8), dtype=x.dtype, device=x.device)[:, 1:1 + h, :d]
    elif how == "heads_out":
        y = torch.empty((x.shape[1], x.shape[0], x.shape[2]), dtype=x.dtype, device=x.device).transpose(0, 1)
    else:
        return x
    y.copy_(x)
    return y


def made(gpu, lens, start, H, Hq, d, page, block, dtype, seed, tail=0, blocks_of=None):
    """Rows, a cache with values everywhere, a shuffled table: block 0 is a cache in 16 bits."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + tail
    q, k, v = (torch.randn((T, h, d), generator=g).to(dtype) for h in (Hq, H, H))
    need = [-(-(s + n) // page) for s, n in zip(start, lens)]
    width = max(need) + 1
    ids = torch.randperm(sum(need) + 2, generator=g).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for j in range(n):
            table[b, j] = ids.pop()
    pool = sum(need) + 2
    if block:
        values = [ref.quantised(torch.randn((pool, H, page, d), generator=g) * 0.3, page // block) for _ in range(2)]
    else:
        values = [(torch.randn((pool, H, page, d), generator=g).to(dtype), None) for _ in range(2)]
    return q, k, v, values, table, T


def offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


CASES = [
    # lens, start, Hq, H, d, page, block, dim, interleaved, dtype
    ([1], [0], 1, 1, 64, 16, 0, 64, False, torch.bfloat16),
    ([1, 0, 3, 40], [5, 9, 0, 30], 6, 3, 64, 16, 0, 32, True, torch.float16),
    ([7, 130], [250, 1], 32, 8, 128, 64, 0, 128, False, torch.bfloat16),
    ([2, 5], [0, 17], 5, 1, 128, 256, 0, 48, False, torch.float16),
    ([1], [0], 1, 1, 64, 16, 16, 64, False, torch.bfloat16),
    ([1, 1, 1], [15, 16, 17], 4, 4, 128, 16, 16, 128, False, torch.float16),
    ([1, 0, 3, 40], [5, 9, 0, 30], 6, 3, 64, 32, 16, 32, True, torch.bfloat16),
    ([7, 130, 1], [250, 1, 63], 8, 2, 128, 64, 64, 128, False, torch.bfloat16),
    ([200, 64], [3, 64], 7, 7, 64, 128, 32, 16, True, torch.float16),
    ([300, 1], [100, 130], 2, 2, 128, 128, 128, 80, False, torch.bfloat16),
    ([600, 9], [1, 250], 3, 1, 128, 256, 256, 128, True, torch.bfloat16),
    ([300], [0], 2, 2, 64, 256, 256, 64, False, torch.float16),
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
@pytest.mark.parametrize("how", ["plain", "wide", "heads_out"])
def test_rotary_append(gpu, case, how):
    lens, start, Hq, H, d, page, block, dim, inter, dtype = case
    q, k, v, values, table, T = made(gpu, lens, start, H, Hq, d, page, block, dtype, seed=len(lens) * 100 + d, tail=3)
    angles = api.rotary_angles(max(s + n for s, n in zip(start, lens)) + 1, dim, device=gpu)
    cu = ints(offsets(lens), gpu)
    kc, vc = (x[0].to(gpu) for x in values)
    ks, vs = (x[1].to(gpu) if block else None for x in values)
    qd, kd, vd = (strided(x.to(gpu), how) for x in (q, k, v))
    qo = strided(torch.full((T, Hq, d), 7.0, dtype=dtype, device=gpu), how)
    ko = strided(torch.full((T, H, d), 7.0, dtype=dtype, device=gpu), how)
    got = api.rotary_append(qd, kd, vd, kc, vc, table.to(gpu), ints(start, gpu), cu, angles, interleaved=inter, q_out=qo,
                            k_out=ko, k_scale=ks, v_scale=vs)
    assert got[0] is qo and got[1] is ko
    n = sum(lens)
    at = [s + i for s, m in zip(start, lens) for i in range(m)]
    tq, tk = ref.rotated(q[:n], angles, at, inter), ref.rotated(k[:n], angles, at, inter)
    # one rounding of the same fp32 values: equal
    assert torch.equal(qo[:n].cpu(), tq.to(dtype)) and torch.equal(ko[:n].cpu(), tk.to(dtype))
    assert bool((qo[n:] == 7).all()) and bool((ko[n:] == 7).all())
    for x, (was, scale), now, now_scale in ((tk, values[0], kc, ks), (v[:n].float(), values[1], vc, vs)):
        want = was.clone()
        if block:
            scale = scale.clone()
            ref.append(x, want, scale, table.tolist(), start, lens)
            assert torch.equal(now_scale.cpu(), scale)
            assert torch.equal(now.cpu().view(torch.uint8), want.view(torch.uint8))
        else:
            for b, m in enumerate(lens):
                for i in range(m):
                    p = start[b] + i
                    want[int(table[b, p // page]), :, p % page] = x[offsets(lens)[b] + i].to(dtype)
            assert torch.equal(now.cpu(), want)
    assert api.device_status(gpu)[0] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,dim,inter", [(64, 64, False), (128, 32, True), (128, 112, False)])
def test_rotary_alone_and_in_place(gpu, dtype, d, dim, inter):
    g = torch.Generator().manual_seed(d + dim)
    T, Hq, H = 37, 6, 2
    q, k = torch.randn((T, Hq, d), generator=g).to(dtype), torch.randn((T, H, d), generator=g).to(dtype)
    at = torch.randint(0, 5000, (T,), generator=g)
    angles = api.rotary_angles(5000, dim, device=gpu)
    qd, kd = q.to(gpu), k.to(gpu)
    out = api.rotary(qd, kd, angles, at.int().to(gpu), interleaved=inter)
    tq, tk = ref.rotated(q, angles, at.numpy(), inter).to(dtype), ref.rotated(k, angles, at.numpy(), inter).to(dtype)
    assert torch.equal(out[0].cpu(), tq) and torch.equal(out[1].cpu(), tk)
    assert torch.equal(qd.cpu(), q)  # the input stays
    both = torch.cat([qd, kd], 1)  # in place, views of one projection
    api.rotary(both[:, :Hq], both[:, Hq:], angles, at.int().to(gpu), interleaved=inter, q_out=both[:, :Hq], k_out=both[:, Hq:])
    assert torch.equal(both.cpu(), torch.cat([tq, tk], 1))


def test_rotation_keeps_products(gpu):
    """What the rotation is for: the product of a rotated query and key depends on the distance alone. fp32 angles
    (off by 2^-25 each) and one bf16 rounding (2^-8) of both sides bound the difference by 2 (2^-8 + 2^-20) |q| |k|."""
    d = 128
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn((1, 1, d), generator=g).bfloat16(), torch.randn((1, 1, d), generator=g).bfloat16()
    angles = api.rotary_angles(9000, d, device=gpu)
    T = 40
    base = torch.arange(T) * 200
    qo, _ = api.rotary(q.expand(T, 1, d).contiguous().to(gpu), k.expand(T, 1, d).contiguous().to(gpu), angles,
                       (base + 31).int().to(gpu))
    _, ko = api.rotary(q.expand(T, 1, d).contiguous().to(gpu), k.expand(T, 1, d).contiguous().to(gpu), angles, base.int().to(gpu))
    s = (qo.double() * ko.double()).sum((1, 2)).cpu()
    bound = 4 * (2.0 ** -8 + 2.0 ** -20) * float(q.double().norm() * k.double().norm())
    assert float((s - s[0]).abs().max()) <= bound


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,page,block", [(64, 32, 16), (128, 64, 64), (128, 128, 128), (64, 256, 32)])
def test_append_picked_rows(gpu, dtype, d, page, block):
    lens, start, H = [5, 0, 1, 33], [60, 3, 31, 0], 3
    _, _, _, values, table, _ = made(gpu, lens, start, H, H, d, page, block, dtype, seed=d)
    g = torch.Generator().manual_seed(9)
    n, drafted = sum(lens), 70
    k, v = (torch.randn((drafted, H, d), generator=g).to(dtype) * 5 for _ in range(2))
    pick = torch.randint(0, drafted, (n,), generator=g)  # the same row twice is fine
    kc, vc = (x[0].to(gpu) for x in values)
    ks, vs = (x[1].to(gpu) for x in values)
    api.cache_append(k.to(gpu), v.to(gpu), kc, vc, table.to(gpu), ints(start, gpu), ints(offsets(lens), gpu),
                     rows=pick.int().to(gpu), k_scale=ks, v_scale=vs)
    for x, (was, scale), now, now_scale in ((k, values[0], kc, ks), (v, values[1], vc, vs)):
        ref.append(x.float(), was, scale, table.tolist(), start, lens, rows=pick.tolist())
        assert torch.equal(now_scale.cpu(), scale)
        assert torch.equal(now.cpu().view(torch.uint8), was.view(torch.uint8))
    assert api.device_status(gpu)[0] == 0


def test_token_by_token_and_at_once(gpu):
    """A block that grows token by token ends with the scale that it has when written at once, and with values off by
    half a step (2^-4) of each rounding on the way at most: one for the first and one a growth of the scale."""
    H, d, page, n = 2, 64, 64, 64
    g = torch.Generator().manual_seed(4)
    x = torch.randn((n, H, d), generator=g) * torch.exp2(torch.arange(n) / 9.0)[:, None, None]
    x = x.bfloat16()
    xd = x.to(gpu)
    table = ints([[0]], gpu)
    caches = []
    for step in (1, n):
        kc = torch.zeros((1, H, page, d), device=gpu).to(E4M3)
        vc, ks, vs = kc.clone(), torch.ones((1, H, 1), device=gpu), torch.ones((1, H, 1), device=gpu)
        for i in range(0, n, step):
            api.cache_append(xd[i:i + step], xd[i:i + step], kc, vc, table, ints([i], gpu), ints([0, step], gpu), k_scale=ks,
                             v_scale=vs)
        caches.append((kc.cpu(), ks.cpu(), vc.cpu(), vs.cpu()))
    (a, sa, av, sav), (b, sb, bv, sbv) = caches
    assert torch.equal(sa, sb) and torch.equal(sav, sa) and torch.equal(sbv, sb)
    assert torch.equal(a.view(torch.uint8), av.view(torch.uint8)) and torch.equal(b.view(torch.uint8), bv.view(torch.uint8))
    want = x.double().transpose(0, 1)
    da, db = (ref.dequantised(y, s)[0] for y, s in ((a, sa), (b, sb)))
    least = 2.0 ** -10 * sb[0].double()[:, :, None]  # half of the smallest step
    assert bool(((db - want).abs() <= 2.0 ** -4 * want.abs() + least).all())
    # restating by powers of two rounds only what falls below the normal range (2^-6 of the scale): half a smallest
    # step each time, at scales that at least double: twice the last one in all
    assert bool(((da - want).abs() <= 2.0 ** -4 * want.abs() + 3 * least).all())


def test_values_that_are_not_finite(gpu):
    H, d, page = 1, 64, 16
    x = torch.ones((3, H, d)).bfloat16()
    x[0, 0, 3], x[1, 0, 4], x[2, 0, 5], x[2, 0, 6] = math.inf, -math.inf, math.nan, 300.0
    kc = torch.zeros((1, H, page, d), device=gpu).to(E4M3)
    vc, ks, vs = kc.clone(), torch.ones((1, H, 1), device=gpu), torch.full((1, H, 1), math.nan, device=gpu)
    z = torch.zeros((3, H, d)).bfloat16()
    api.cache_append(x.to(gpu), z.to(gpu), kc, vc, ints([[0]], gpu), ints([0], gpu), ints([0, 3], gpu), k_scale=ks, v_scale=vs)
    got = ref.dequantised(kc.cpu(), ks.cpu())[0, 0, :3]
    assert float(ks) == 1.0  # 300 needs 2^0
    assert torch.equal(torch.isnan(got), ~torch.isfinite(x[:, 0]))
    fine = torch.isfinite(x[:, 0])
    assert bool(((got - x[:, 0].double())[fine].abs() <= 2.0 ** -4 * x[:, 0].double()[fine].abs()).all())
    assert float(vs) == 2.0 ** -118 and bool((vc.float() == 0).all())
    # a scale that is none: the new tokens' own, what is there stays
    vs.fill_(math.nan)
    before = vc.clone()
    api.cache_append(x.to(gpu), x.to(gpu), kc, vc, ints([[0]], gpu), ints([5], gpu), ints([0, 3], gpu), k_scale=ks, v_scale=vs)
    assert float(vs) == 1.0 and torch.equal(vc[:, :, :5].view(torch.uint8), before[:, :, :5].view(torch.uint8))


@pytest.mark.parametrize("eight", [False, True])
def test_what_lies_outside_is_left_out(gpu, eight):
    """Positions outside the angles or the table, pages outside the cache: recorded, left out, the rest as it should be."""
    H, Hq, d, page, dtype = 2, 4, 64, 16, torch.bfloat16
    g = torch.Generator().manual_seed(3)
    lens, start = [2, 2, 2, 2], [0, 30, 16, -1]  # the second runs past the table, the third's page is -1, the fourth starts early
    T = sum(lens)
    q, k, v = (torch.randn((T, h, d), generator=g).to(dtype).to(gpu) for h in (Hq, H, H))
    table = ints([[0, 1], [2, 3], [4, -1], [5, 6]], gpu)
    kc = torch.zeros((7, H, page, d), device=gpu).to(E4M3 if eight else dtype)
    vc = kc.clone()
    ks = torch.full((7, H, 1), 3.0, device=gpu) if eight else None
    vs = None if ks is None else ks.clone()
    angles = api.rotary_angles(32, d, device=gpu)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    api.rotary_append(q, k, v, kc, vc, table, ints(start, gpu), ints(offsets(lens), gpu), angles, q_out=qo, k_out=ko,
                      k_scale=ks, v_scale=vs)
    assert api.device_status(gpu)[0] == 6
    at = [0, 1, 30, 31, 16, 17, -1, 0]
    ok = [i for i in range(T) if at[i] >= 0]
    want = ref.rotated(q.cpu()[ok], angles, [at[i] for i in ok], False).to(dtype)
    assert torch.equal(qo.cpu()[ok], want)
    assert bool((qo[6] == 7).all()) and bool((ko[6] == 7).all())  # position -1
    written = {(0, 0), (0, 1), (3, 14), (3, 15), (5, 0)}
    for p in range(7):
        for i in range(page):
            assert bool((vc.float()[p, :, i] != 0).any()) == ((p, i) in written), (p, i)
    # positions of their own, one outside
    places = ints([3, 5, 31, 32, 0, 1, 2, -4], gpu)
    qo.fill_(7.0)
    api.rotary(q, k, angles, places, q_out=qo, k_out=ko)
    assert api.device_status(gpu)[0] == 6
    assert bool((qo[3] == 7).all()) and bool((qo[7] == 7).all()) and not bool((qo[2] == 7).any())
    # decreasing offsets
    api.rotary_append(q, k, v, kc, vc, table, ints([0] * 4, gpu), ints([0, 4, 2, 6, 9], gpu), angles, k_scale=ks, v_scale=vs)
    assert api.device_status(gpu)[0] == 6


def test_large_strides_and_offsets(gpu):
    """Pages and planes of which the offsets pass 32 bits: a pool of 2^33 bytes, of which the last pages are used."""
    H, d, page, dtype = 1, 128, 256, torch.bfloat16
    pool = (1 << 33) // (H * page * d) + 3
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn((20, H, d), generator=g).to(dtype) for _ in range(2))
    kc = torch.empty((pool, H, page, d), dtype=E4M3, device=gpu)
    vc = torch.empty_like(kc)
    ks, vs = torch.ones((pool, H, 4), device=gpu), torch.ones((pool, H, 4), device=gpu)
    table = ints([[pool - 1, pool - 2]], gpu)
    api.cache_append(k.to(gpu), v.to(gpu), kc, vc, table, ints([250], gpu), ints([0, 20], gpu), k_scale=ks, v_scale=vs)
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        got = torch.cat([ref.dequantised(c[pool - 1:].cpu(), s[pool - 1:].cpu())[0, :, 250:],
                         ref.dequantised(c[pool - 2:pool - 1].cpu(), s[pool - 2:pool - 1].cpu())[0, :, :14]], 1)
        want = x.double().transpose(0, 1)
        assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10).all())
    assert api.device_status(gpu)[0] == 0


def test_captured_and_replayed_with_other_lengths(gpu):
    H, Hq, d, page, dtype = 2, 4, 128, 64, torch.bfloat16
    g = torch.Generator().manual_seed(5)
    T = 24
    q, k, v = (torch.randn((T, h, d), generator=g).to(dtype).to(gpu) for h in (Hq, H, H))
    angles = api.rotary_angles(400, d, device=gpu)
    table = ints([[0, 1, 2], [3, 4, 5]], gpu)
    start, cu = ints([5, 100], gpu), ints([0, 4, T], gpu)
    caches = [torch.zeros((6, H, page, d), device=gpu).to(E4M3) for _ in range(2)]
    scales = [torch.ones((6, H, 2), device=gpu) for _ in range(2)]
    qo, ko = torch.empty_like(q), torch.empty_like(k)

    def call():
        api.rotary_append(q, k, v, *caches, table, start, cu, angles, q_out=qo, k_out=ko, k_scale=scales[0], v_scale=scales[1])

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, at in (([4, 20], [5, 100]), ([24, 0], [0, 7]), ([1, 3], [63, 64])):
        for c, s in zip(caches, scales):
            c.copy_(torch.zeros(c.shape, device=gpu).to(E4M3))
            s.fill_(1.0)
        start.copy_(ints(at, gpu))
        cu.copy_(ints(offsets(lens), gpu))
        graph.replay()
        x = ref.rotated(k.cpu()[:sum(lens)], angles, [a + i for a, n in zip(at, lens) for i in range(n)], False)
        want, scale = torch.zeros((6, H, page, d)).to(E4M3), torch.ones((6, H, 2))
        ref.append(x, want, scale, table.tolist(), at, lens)
        assert torch.equal(scales[0].cpu(), scale) and torch.equal(caches[0].cpu().view(torch.uint8), want.view(torch.uint8))
    assert api.device_status(gpu)[0] == 0


def test_wrapper_refusals(gpu):
    dtype, d, H = torch.bfloat16, 64, 2
    q, k, v = (torch.zeros((4, h, d), dtype=dtype, device=gpu) for h in (4, H, H))
    kc = torch.zeros((4, H, 32, d), device=gpu).to(E4M3)
    vc, ks = kc.clone(), torch.ones((4, H, 2), device=gpu)
    table, start, cu = ints([[0, 1]], gpu), ints([0], gpu), ints([0, 4], gpu)
    angles = api.rotary_angles(64, d, device=gpu)
    ok = dict(q=q, k=k, v=v, k_cache=kc, v_cache=vc, table=table, start=start, cu=cu, angles=angles, k_scale=ks, v_scale=ks.clone())
    api.rotary_append(**ok)
    for bad in (dict(k_scale=None), dict(v_scale=None), dict(k_scale=ks.double()), dict(k_scale=ks[:, :, :1]),
                dict(k_scale=torch.ones((4, H, 3), device=gpu), v_scale=torch.ones((4, H, 3), device=gpu)),
                dict(k_scale=ks.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(k_cache=kc.to(dtype), v_cache=vc.to(dtype)), dict(k_cache=kc[:, :, :, :32]),
                dict(q=q[:, :3]), dict(k=k.half()), dict(v=v[:3]), dict(angles=angles.double()), dict(angles=angles[:, :24]),
                dict(angles=angles.t()), dict(positions=torch.zeros(3, dtype=torch.int32, device=gpu)),
                dict(positions=torch.zeros(4, device=gpu)), dict(q_out=q[:, :, :32]), dict(k_out=k.half()),
                dict(start=start.long()), dict(cu=cu.long()), dict(table=table.long()), dict(q=q.float()),
                dict(q=q.cpu()), dict(k_scale=ks.cpu())):
        with pytest.raises(ValueError):
            api.rotary_append(**{**ok, **bad})
    with pytest.raises(ValueError):
        api.rotary(q, k, angles, None)
    with pytest.raises(ValueError):  # scales of a cache in 16 bits
        api.cache_append(k, v, kc.to(dtype), vc.to(dtype), table, start, cu, k_scale=ks, v_scale=ks)
