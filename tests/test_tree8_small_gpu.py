"""How far attention over a cache in 8 bits rounds probabilities that are small beside the row's largest.

P is formed 2^11 times its value in fp16 with few rows a sequence and 2^9 times with many, less up to one bit that the
reference of the values' scales may be above the largest of them; fp16 below 2^-14 is off by 2^-25. With few rows it is
then split into e5m2, three parts in bf16 and four in fp16: enumerated over all fp16 numbers, the sum of the parts is exact
but for 2^-21 below 2^-10 and 2^-23 below 2^-12. So the product of a probability and a scale is off by half a step of the type, or by
  2 (2^-21 + 2^-25) 2^-11 = 1.0625 2^-31, 2 (2^-23 + 2^-25) 2^-11 = 1.25 2^-33 and 2 2^-25 2^-9 = 2^-33
of the product of the row's largest probability and the largest scale.
"""

import math

import numpy as np
import pytest
import torch

from io_aware_exact_04_gb300 import api
from tests import serving_ref
from tests.test_tree8_gpu import BF16, E4M3, FP16, ints

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dtype", [BF16, FP16])
KINDS = pytest.mark.parametrize("n,G", [(1, 2), (2, 4), (2, 8), (16, 8)], ids=["few4", "few8", "few16", "many"])


def floor_of(dtype, n, G):
    if n * G > 16:
        return 2.0 ** -33
    return 1.0625 * 2.0 ** -31 if dtype is BF16 else 1.25 * 2.0 ** -33


@TYPES
@KINDS
@pytest.mark.parametrize("d", [64, 128])
def test_a_small_probability_alone(gpu, dtype, n, G, d):
    """Two cached tokens a sequence: one with nearly all of the weight and no value, the other 2^-x of it, x from 0 to 34."""
    B, scale, vscale = 64, d ** -0.5, 2.0 ** 7
    T = n * B
    q = torch.zeros((T, G, d), device=gpu)
    q[:, :, 3] = torch.linspace(2.0 ** -6, 8.0, T * G, device=gpu).view(T, G)
    q = q.to(dtype)
    k = torch.zeros((T, 1, d), dtype=dtype, device=gpu)
    kc, vc = (torch.zeros((B, 1, 16, d), dtype=torch.uint8, device=gpu) for _ in range(2))
    kc[:, 0, 0, 3], vc[:, 0, 1] = 0x38, 0x7E  # 1.0 and 448
    kscale = (torch.linspace(0.9, 1.0, B, device=gpu) * (34 * math.log(2) / (8.0 * scale))).view(B, 1, 1)
    vs = torch.full((B, 1, 1), vscale, device=gpu)
    mask = torch.zeros((T, 1), dtype=torch.int32, device=gpu)  # no node sees another
    o, lse = api.forward_tree(q, k, k, kc.view(E4M3), vc.view(E4M3), ints([[b] for b in range(B)], gpu), ints([2] * B, gpu),
                              ints(serving_ref.offsets([n] * B), gpu), mask=mask, scale=scale, k_scale=kscale, v_scale=vs)
    assert api.device_status(gpu)[0] == 0
    s = q[:, :, 3].double() * kscale.double().view(B, 1).repeat_interleave(n, 0) * scale
    p = 1.0 / (1.0 + torch.exp(s))
    value, unit = 448.0 * vscale, serving_ref.UNIT[dtype]
    want, biggest = p * value, 1.0 - p
    delta = d * 2.0 ** -23 * s + 2.0 ** -19
    bound = (2 * unit + 2 * delta) * want + floor_of(dtype, n, G) * biggest.clamp(min=0.5) * value + 2.0 ** -25
    off = (o.double() - want[:, :, None]).abs()
    assert torch.isfinite(o).all() and bool((off <= bound[:, :, None]).all()), float((off / bound[:, :, None]).max())
    assert float(want.min()) < 2.0 ** -29 * value and float(want.max()) > 0.4 * value


@TYPES
@KINDS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("large", [0, 8, 16])
def test_nodes_beside_a_large_scale(gpu, dtype, n, G, d, large):
    """A cached token that is hardly seen, with a scale of 2^large: the nodes' values, which are of size 1, are rounded
    with it in mind where the kernel takes both into the same sum."""
    B, scale, S = 64, d ** -0.5, 2.0 ** large
    T = n * B
    g = torch.Generator(device=gpu).manual_seed(5)
    q = torch.ones((T, G, d), device=gpu).to(dtype)
    k = torch.zeros((T, 1, d), dtype=dtype, device=gpu)
    v = torch.randn((T, 1, d), generator=g, device=gpu).to(dtype)
    kc, vc = (torch.zeros((B, 1, 16, d), dtype=torch.uint8, device=gpu) for _ in range(2))
    kc[:, 0, 0], vc[:, 0, 0] = 0xB8, 0x38  # -1.0 and 1.0
    kscale = torch.full((B, 1, 1), 40.0 * math.log(2) / (d * scale), device=gpu)
    vs = torch.full((B, 1, 1), S, device=gpu)
    args = (q, k, v, kc.view(E4M3), vc.view(E4M3), ints([[b] for b in range(B)], gpu), ints([1] * B, gpu),
            ints(serving_ref.offsets([n] * B), gpu))
    o, lse = api.forward_tree(*args, scale=scale, k_scale=kscale, v_scale=vs)
    assert api.device_status(gpu)[0] == 0
    x = np.float32(40.0 * math.log(2) / (d * scale))
    pc = math.exp(-float(x) * d * scale)
    unit = serving_ref.UNIT[dtype]
    # stored: what a node's value is held as, beside its scale
    few = n * G <= 16
    stored = 2.0 ** 15 if not few and dtype is BF16 else 8.0
    top = max(S, 1.0) if not few else 1.0
    for b in range(B):
        vv = v[b * n:(b + 1) * n, 0].double()
        for i in range(n):
            total = (i + 1) + pc
            want = (vv[: i + 1].sum(0) + pc * S) / total
            mag = (vv[: i + 1].abs().sum(0) + pc * S) / total
            bound = (unit + 2 * 2.0 ** -18) * mag + unit * want.abs() + floor_of(dtype, n, G) * top * stored + 2.0 ** -25
            off = (o[b * n + i].double() - want).abs()
            assert bool((off <= bound).all()), float((off / bound).max())
