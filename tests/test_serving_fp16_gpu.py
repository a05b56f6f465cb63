"""fp16: probabilities far below the largest one still count. One key takes nearly all of the weight, with a
value of zero (an attention sink), and thousands of others share the rest.
"""

import pytest
import torch

import serving_ref as ref
from io_aware_exact_04_gb300 import api
from test_serving_gpu import Cache, ints, ok

pytestmark = pytest.mark.gpu


def sink_rows(n, Hkv, d, at, nats, device, dtype, seed):
    """Keys and values of n tokens: scores are the keys' first elements times the query's, so exact."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    k = torch.zeros((n, Hkv, d), dtype=torch.float32, device=device)
    k[:, :, 0] = torch.randint(-64, 65, (n, Hkv), generator=g, device=device) / 256
    v = torch.randn((n, Hkv, d), generator=g, device=device) * 0.5 + 0.5
    k[at, :, 0], v[at] = nats, 0.0
    return k.to(dtype), v.to(dtype)


def bound(o, p_v, v_sum, unit):
    """Scores are exact products, times log2(e) in fp32 and less the maximum: below 26 they are off by less than
    2^-18 in all, the exponential by 2^-22 of its value. l and O are fp32 sums of at most 512 steps' (64 keys each),
    a step off by 2^-24 of l and 2^-23 of O (which may be cut, not rounded): delta = 2^-14 holds all of it. P for
    the product is off by half a step, or where it is subnormal by half of the smallest one, 2^-25, at 2^9 times
    its value: 2^-34 of the largest, which is 1 here. O is rounded once, by half of 2^-24 at least."""
    delta = 2.0 ** -14
    return (unit + 2 * delta) * p_v + 2.0 ** -34 * v_sum + unit * o.abs() + 2.0 ** -25


def exact(q, k, v, seen):
    """O, sum p |v| and sum |v| in 64 bits: q [n, d], k and v [m, d]."""
    s = torch.where(seen, q.double() @ k.double().t(), float("-inf"))
    p = torch.softmax(s, 1)
    return p @ v.double(), p @ v.double().abs(), torch.where(seen, 1.0, 0.0).double() @ v.double().abs()


def compare(o, lse, q, k, v, rows, seen_of, G, dtype):
    """rows: tokens compared; seen_of(i): how many keys token i sees (a prefix)."""
    worst = 0.0
    for h in range(q.shape[1]):
        kk, vv = k[:, h // G], v[:, h // G]
        seen = torch.arange(k.shape[0], device=q.device)[None, :] < torch.tensor([seen_of(i) for i in rows], device=q.device)[:, None]
        want, p_v, v_sum = exact(q[rows, h], kk, vv, seen)
        tol = bound(want, p_v, v_sum, ref.UNIT[dtype])
        worst = max(worst, float(((o[rows, h].double() - want).abs() / tol).max()))
        s = torch.where(seen, q[rows, h].double() @ kk.double().t(), float("-inf"))
        assert float((lse[h, rows].double() - torch.logsumexp(s, 1)).abs().max()) <= 2.0 ** -14
    assert worst <= 1.0, f"O off by {worst} times its bound"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("nats", [12.0, 17.0, 17.5])
@pytest.mark.parametrize("d,G,at", [(64, 1, 0), (64, 4, 20000), (64, 20, 0), (128, 4, 0), (128, 8, 32766), (128, 24, 5000)])
def test_decoding_beside_a_sink(gpu, d, G, at, nats, dtype):
    """One token over 32767 cached ones, with up to and with more than 16 rows."""
    L, Hkv = 32767, 2
    k, v = sink_rows(L + 1, Hkv, d, at, nats, gpu, dtype, seed=d + G)
    c = Cache([0], Hkv, 64, d, dtype, gpu, width=512, extra=512)
    table = torch.randperm(512, generator=torch.Generator().manual_seed(1)).to(torch.int32)[None].to(gpu)
    for x, plane in ((k, 0), (v, 1)):
        pages = torch.cat([x[:L], torch.full_like(x[:1], float("nan"))]).unflatten(0, (512, 64)).transpose(1, 2)
        c.kv[plane, table[0].long()] = pages
    q = torch.zeros((1, G * Hkv, d), dtype=dtype, device=gpu)
    q[:, :, 0] = 1.0
    o, lse = api.forward_tree(q, k[L:], v[L:], c.kv[0], c.kv[1], table, ints([L], gpu), ints([0, 1], gpu), scale=1.0)
    ok(gpu)
    compare(o, lse, q, k, v, [0], lambda i: L + 1, G, dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("nats", [14.0, 17.0])
@pytest.mark.parametrize("d,G,at", [(64, 1, 0), (64, 3, 700), (128, 2, 0), (128, 16, 130)])
def test_prompts_beside_a_sink(gpu, d, G, at, nats, dtype):
    n, Hkv = 8000, 2
    k, v = sink_rows(n, Hkv, d, at, nats, gpu, dtype, seed=d + G)
    q = torch.zeros((n, G * Hkv, d), dtype=dtype, device=gpu)
    q[:, :, 0] = 1.0
    o, lse = api.forward_prompt(q, k, v, ints([0, n], gpu), scale=1.0)
    ok(gpu)
    rows = [0, 1, 63, 64, 127, 128, 129, 500, 701, 1000, 4097, 7998, 7999]
    compare(o, lse, q, k, v, rows, lambda i: i + 1, G, dtype)
