"""Appends into a cache in 8 bits where a block's scale grows, or is not one of the library's, at every block size, by
few tokens and by many: bytes and scales are those of the plain form."""

import math

import pytest
import torch

from io_aware_exact_04_gb300 import api
from tests import cache8_ref as ref
from tests.test_rotary_gpu import ints, made, offsets

pytestmark = pytest.mark.gpu
MANY, FEW = ([70, 300, 33, 0, 18], [13, 3, 250, 5, 31]), ([1, 5, 0, 3, 20], [13, 3, 250, 31, 40])


def appended(gpu, k, v, values, table, start, lens, **rotary):
    kc, vc = (x[0].to(gpu) for x in values)
    ks, vs = (x[1].to(gpu) for x in values)
    args = (kc, vc, table.to(gpu), ints(start, gpu), ints(offsets(lens), gpu))
    out = k.to(gpu)
    if rotary:  # in place
        q = torch.ones_like(out)
        api.rotary_append(q, out, v.to(gpu), *args, q_out=q, k_out=out, k_scale=ks, v_scale=vs, **rotary)
    else:
        api.cache_append(out, v.to(gpu), *args, k_scale=ks, v_scale=vs)
    assert api.device_status(gpu)[0] == 0
    return out, (kc, ks), (vc, vs)


def same(got, want):
    values, scales = want
    assert torch.equal(got[1].cpu(), scales), "scales"
    assert torch.equal(got[0].cpu().view(torch.uint8), values.view(torch.uint8)), "elements"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,start", [MANY, FEW], ids=["many", "few"])
@pytest.mark.parametrize("d,page,block", [(d, max(32, b), b) for d in (64, 128) for b in (16, 32, 64, 128, 256)])
def test_blocks_that_grow(gpu, dtype, lens, start, d, page, block):
    H = 3
    _, k, v, values, table, _ = made(gpu, lens, start, H, H, d, page, block, dtype, seed=block + d)
    size = torch.exp2(torch.arange(sum(lens)).float() % 23 - 11)[:, None, None]  # larger and smaller than what is there
    k, v = ((x.float() * size).to(dtype) for x in (k, v))
    angles = api.rotary_angles(600, d, device=gpu)
    at = [s + i for s, n in zip(start, lens) for i in range(n)]
    for rotary in ({}, dict(angles=angles)):
        out, got_k, got_v = appended(gpu, k, v, values, table, start, lens, **rotary)
        turned = ref.rotated(k, angles, at, False) if rotary else k.float()
        if rotary:
            assert torch.equal(out.cpu(), turned.to(dtype))
        for x, (was, scale), got in ((turned, values[0], got_k), (v.float(), values[1], got_v)):
            want = (was.clone(), scale.clone())
            ref.append(x, *want, table.tolist(), start, lens)
            same(got, want)


@pytest.mark.parametrize("lens,start", [MANY, FEW], ids=["many", "few"])
@pytest.mark.parametrize("block", [16, 64])
def test_scales_of_another_making(gpu, lens, start, block):
    """No powers of two, ones at the ends of the range, and what is no scale at all."""
    dtype, d, H, page = torch.bfloat16, 128, 4, 64
    _, k, v, values, table, _ = made(gpu, lens, start, H, H, d, page, block, dtype, seed=3)
    odd = torch.tensor([1.3, 0.7, 2.0 ** -126, 2.0 ** -120, 2.0 ** -118, 2.0 ** 119, 2.0 ** 121, 3e38, 0.0, -1.0, math.nan,
                        math.inf, 1e-40, 1.9999999, 0.01, 1.0])
    for i, (was, scale) in enumerate(values):
        scale.copy_(odd[(torch.arange(scale.numel()) * 7 + i).remainder(len(odd))].view(scale.shape))
    k = (k.float() * 2.0 ** -20).to(dtype)
    _, got_k, got_v = appended(gpu, k, v, values, table, start, lens)
    for x, (was, scale), got in ((k, values[0], got_k), (v, values[1], got_v)):
        want = (was.clone(), scale.clone())
        ref.append(x.float(), *want, table.tolist(), start, lens)
        assert torch.equal(got[1].cpu().nan_to_num(-7.0), want[1].nan_to_num(-7.0))
        assert torch.equal(got[0].cpu().view(torch.uint8), want[0].view(torch.uint8))
