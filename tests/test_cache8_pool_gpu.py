"""Pools in 8 bits: update and compact move pages with their scales."""

import random

import pytest
import torch

from io_aware_exact_04_gb300 import api
from tests import serving_ref

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def pool(gpu, planes, n, H, page, d, block, slots, width, used, seed):
    r = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    kv = torch.randint(0, 256, (planes, n, H, page, d), generator=g, dtype=torch.uint8)
    scales = torch.randn((planes, n, H, page // block), generator=g)
    ids = r.sample(range(n), n)
    lens, table = [], []
    for _ in range(slots):
        k = r.randrange(0, min(width, len(ids), max(1, used)) + 1)
        row = [ids.pop() for _ in range(k)]
        lens.append(0 if k == 0 else (k - 1) * page + r.randrange(1, page + 1))
        table.append(row + [-1] * (width - k))
    return r, kv, scales, lens, table


@pytest.mark.parametrize("planes,H,page,d,block", [(1, 1, 16, 64, 16), (4, 3, 32, 128, 16), (2, 2, 64, 64, 64), (3, 5, 256, 128, 32)])
@pytest.mark.parametrize("seed", range(3))
def test_update(gpu, planes, H, page, d, block, seed):
    n, slots, width = 40, 6, 6
    r, kv, scales, lens, table = pool(gpu, planes, n, H, page, d, block, slots, width, 4, seed)
    src = [r.randrange(slots) if r.random() < 0.6 else s for s in range(slots)]
    new = [min(width * page, max(0, lens[src[s]] + r.choice([-7, 0, 1, page]))) if r.random() < 0.8 else 0 for s in range(slots)]
    kd, sd = kv.to(gpu).view(E4M3), scales.to(gpu)
    td, ld = (torch.tensor(x, dtype=torch.int32, device=gpu) for x in (table, lens))
    info = api.cache_update(kd, td, ld, *(torch.tensor(x, dtype=torch.int32, device=gpu) for x in (src, new)), scales=sd)
    want_kv, want_s = kv.clone(), scales.clone()
    made, want_lens, want_info = serving_ref.update(want_kv, table, lens, src, new, page)
    assert info.tolist() == want_info and td.tolist() == made and ld.tolist() == want_lens
    assert torch.equal(kd.view(torch.uint8).cpu(), want_kv)
    # the scales follow as a cache of one value a block would, with the lengths in blocks
    keep = [min(new[s], lens[src[s]]) for s in range(slots)]
    for s in range(slots):
        j, part = keep[s] // page, keep[s] % page
        if part and made[s][j] != table[src[s]][j]:
            w = -(-part // block)
            want_s[:, made[s][j], :, :w] = scales[:, table[src[s]][j], :, :w]
    assert torch.equal(sd.cpu(), want_s)
    assert api.device_status(gpu)[0] == 0


@pytest.mark.parametrize("planes,H,page,d,block", [(1, 1, 16, 64, 16), (4, 3, 32, 128, 16), (2, 40, 64, 64, 16)])
@pytest.mark.parametrize("seed", range(2))
def test_compact(gpu, planes, H, page, d, block, seed):
    n, slots, width = 33, 5, 5
    _, kv, scales, lens, table = pool(gpu, planes, n, H, page, d, block, slots, width, 4, seed + 50)
    kd, sd = kv.to(gpu).view(E4M3), scales.to(gpu)
    td, ld = (torch.tensor(x, dtype=torch.int32, device=gpu) for x in (table, lens))
    info = api.cache_compact(kd, td, ld, scales=sd)
    want_kv, want_s = kv.clone(), scales[:, :, :, :, None].clone()
    made, want_info = serving_ref.compact(want_kv, table, lens, page)
    serving_ref.compact(want_s, table, lens, page)
    assert info.tolist() == want_info and td.tolist() == made
    assert torch.equal(kd.view(torch.uint8).cpu(), want_kv) and torch.equal(sd.cpu(), want_s[..., 0])
    assert api.device_status(gpu)[0] == 0


def test_planes_apart_and_refusals(gpu):
    """Planes that are views of a wider pool; and what the wrapper refuses."""
    big = torch.zeros((4, 8, 2, 16, 64), dtype=torch.uint8, device=gpu)
    big[0, 7] = 5
    scales = torch.zeros((4, 8, 2, 1), device=gpu)
    scales[0, 7] = 9.0
    table, lens = torch.tensor([[7]], dtype=torch.int32, device=gpu), torch.tensor([3], dtype=torch.int32, device=gpu)
    api.cache_compact(big[::2].view(E4M3), table, lens, scales=scales[::2])
    assert table.tolist() == [[0]] and bool((big[0, 0] == 5).all()) and bool((scales[0, 0] == 9).all())
    assert bool((big[1] == 0).all()) and bool((scales[1] == 0).all())
    for bad in (None, scales[:1], scales.double(), scales[:, :, :, :0], scales.cpu(),
                scales[:, :, :1], torch.zeros((8, 4, 2, 1), device=gpu).transpose(0, 1)):
        with pytest.raises((ValueError, RuntimeError)):
            api.cache_compact(big.view(E4M3), table, lens, scales=bad)
    with pytest.raises(ValueError):
        api.cache_compact(big.view(torch.float16), table, lens, scales=scales)
