"""tcgen05 in 8 bits: every operand layout that the attention over an 8-bit cache uses, and how it sums."""

import ctypes

import pytest
import torch

from io_aware_exact_04_gb300 import _lib

pytestmark = pytest.mark.gpu


def product(gpu, a, b, N, d, a_mn, e5m2, b_mn=0, b_from=0):
    status = torch.zeros(4, dtype=torch.int32, device=gpu)
    out = torch.full((128, N), float("nan"), device=gpu)
    a, b = a.to(gpu), b.to(gpu)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    rc = _lib.load("libfa_selftest.so").fa_selftest_mma8(p(a), p(b), p(out), N, d, a_mn, e5m2, b_mn, b_from,
                                                         p(status),
                                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0, 0, 0]
    return out.cpu().double()[: d if a_mn else 128]


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("a_mn", [0, 1])
@pytest.mark.parametrize("e5m2", [0, 1])
@pytest.mark.parametrize("N", [32, 96, 256])
def test_operand_layouts(gpu, d, a_mn, e5m2, N):
    g = torch.Generator().manual_seed(d + N)
    K = 128 if a_mn else d
    a = torch.randint(-6, 7, (128, d), generator=g).float().to(torch.float8_e4m3fn)
    b = torch.randint(-3, 4, (N, K), generator=g).float().to(torch.float8_e5m2 if e5m2 else torch.float8_e4m3fn)
    want = (a.double().t() if a_mn else a.double()) @ b.double().t()
    assert torch.equal(product(gpu, a, b, N, d, a_mn, e5m2), want)  # integers: exact in fp32


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("pitch,at,N", [(64, 0, 32), (64, 32, 16), (64, 32, 32), (128, 0, 64), (128, 64, 32), (128, 64, 64),
                                        (128, 0, 128), (64, 0, 64)])
def test_second_operand_by_columns(gpu, d, pitch, at, N):
    """The second operand with its columns next to each other, from a place inside a swizzled row."""
    g = torch.Generator().manual_seed(pitch + at + N)
    a = torch.randint(-6, 7, (128, d), generator=g).float().to(torch.float8_e4m3fn)
    b = torch.randint(-3, 4, (128, pitch), generator=g).float().to(torch.float8_e5m2)
    want = a.double().t() @ b.double()[:, at:at + N]
    assert torch.equal(product(gpu, a, b, N, d, 1, 1, pitch, at), want)


@pytest.mark.parametrize("a_mn", [0, 1])
def test_sums_are_kept_in_32_bits(gpu, a_mn):
    """Products between 2^-12 and 2^17 of either sign: the sum of K of them in fp32, in any order, is off by at most
    K 2^-24 of the sum of their magnitudes (truncated instead of rounded: twice that)."""
    g = torch.Generator().manual_seed(1)
    d = K = 128
    x = torch.randn((128, d), generator=g) * torch.exp2(torch.randint(-4, 8, (128, d), generator=g).float())
    y = torch.randn((64, K), generator=g) * torch.exp2(torch.randint(-4, 8, (64, K), generator=g).float())
    a, b = x.clamp(-440, 440).to(torch.float8_e4m3fn), y.clamp(-440, 440).to(torch.float8_e4m3fn)
    m = a.double().t() if a_mn else a.double()
    got = product(gpu, a, b, 64, d, a_mn, 0)
    off = (got - m @ b.double().t()).abs() / (m.abs() @ b.double().t().abs())
    print("largest error of a sum, relative to its magnitudes: 2^%.1f" % float(torch.log2(off.max())))
    assert float(off.max()) <= K * 2.0 ** -23
